// diffragged_fwd: what its two kernels (d = 64 and d = 128) have in common: how
// the work is cut, how a share of it is walked, the launch, and how a tile's values
// are cleared of what not all rows see.
//
// The mathematics.  Rows are r = (token, query head of the group) of one
// key/value head, 128 to a tile, so that a tile's rows share every key and value
// that it reads:
//   x_m[r, j] = q_m[r] . k_m[j] / sqrt(d),  map_m = softmax_j(x_m),  m = 1, 2
//   o[r] = sum_j (map1[r, j] - lambda_h map2[r, j]) v[j], then the head norm,
// keys j up to the row's position.  An item is a (sequence, key/value head, tile
// of rows) with its keys in tiles of 128; each map is an ordinary softmax with a
// running reference and sum, so that ranges of an item's keys done by different
// CTAs join exactly: with M = max m_s, O = sum_s 2^(m_s - M) O_s, l alike.
//
// How the work is cut.  All items lie on a line, each some steps that stand for
// its end, then some for each key tile (a step is about 0.27 us; a tile of a few
// rows leaves most softmax warps idle and takes less), and every share (a CTA, or
// a pair of them) takes an equal piece of it, found from q_start and kv_len on the
// device: a batch of prompts, chunks and single tokens is balanced, and a
// captured graph replays with others.  A tile belongs to the share with its first
// step.  Items that a border cuts leave partial states that a second kernel
// joins.  Where cutting gains less than that costs, shares take whole items (see
// cut_line).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "debug_check.cuh"
#include "ptx.cuh"
#include "ragged.h"

namespace diffattn {

// An item that a border cuts, as the share with its first tile leaves it for the second kernel.
struct RaggedJoin {
  int32_t parts;  // 0: none
  int32_t slot;   // of the first part; the k-th is in slot 2 (slot / 2 + k)
  int32_t hk, row, tokens, first;  // key/value head, first row and its position, tokens
  int32_t pad[2];
};

struct RaggedParams {
  const int32_t *q_start, *kv_len, *page_table;
  const float *lambda, *norm_w;
  __nv_bfloat16 *out;
  int32_t *status;
  float *part;        // [2 * shares][2 maps][part_floats(2 d)]
  RaggedJoin *joins;  // [shares]
  float *swap;        // d = 128: what the CTAs of a pair hand one another
  int64_t out_n, out_h;  // element strides of a token and a head
  int32_t B, N, kv_heads, group, tokens;  // N: packed rows; tokens: of a tile, 128 / group
  int32_t num_pages, max_pages, page_size, piece_rows;
  int32_t causal, headnorm, shares;
  int32_t group_bits;  // group = 2^group_bits, or -1
  FastDiv by_page, by_group, by_tokens;
  float eps, out_scale, scale_log2;
};

diffattn_status launch_ragged_main_d64(const RaggedParams &p, const CUtensorMap (&maps)[5], bool fp8,
                                       cudaStream_t stream);
diffattn_status launch_ragged_main_d128(const RaggedParams &p, const CUtensorMap (&maps)[5],
                                        bool fp8, cudaStream_t stream);

size_t ragged_swap_bytes(int shares);  // of d = 128

using RaggedKernel = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap,
                              const CUtensorMap, const CUtensorMap, const RaggedParams);
// One launch of a main kernel, `cluster` CTAs a share, behind the kernel before (dependent launch).
// ready: which devices have the kernel's shared memory size set.
inline diffattn_status launch_ragged_kernel(RaggedKernel kernel, std::atomic<bool> (&ready)[64],
                                            const RaggedParams &p, const CUtensorMap (&maps)[5],
                                            int threads, uint32_t smem, int cluster,
                                            cudaStream_t stream) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DIFFATTN_ERR_CUDA;
  if (dev < 0 || dev >= 64) return DIFFATTN_ERR_UNSUPPORTED;
  if (!ready[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem)) != cudaSuccess)
      return DIFFATTN_ERR_CUDA;
    ready[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.shares * cluster));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, maps[0], maps[1], maps[2], maps[3], maps[4], p) ==
                 cudaSuccess
             ? DIFFATTN_OK
             : DIFFATTN_ERR_CUDA;
}

// A part: O [2 d columns][128 rows] as accumulated, references (log2 units), sums.
__host__ __device__ constexpr int64_t part_floats(int dv) { return (dv + 2) * 128ll; }

namespace {

constexpr int kTile = 128;  // keys of a tile, and rows
// Steps, measured at d = 64: a tile takes 1.37 us with 128 rows and 1.08 us with up to 16 (one warp
// of eight has rows), an item 4 us beside its tiles.
constexpr int kTileSteps = 5, kFewSteps = 4, kFewRows = 16, kItemSteps = 15;
// What leaving parts and joining them costs a call, about, and the least that a share is cut to.
constexpr int kJoinSteps = 40, kLeastSteps = 3 * kTileSteps;
// A product adds to O in fp32 and drops the bits that do not fit, so that where a column's terms are of
// one sign O falls behind its sum: by 0.03 to 0.06 % after 2^17 keys, 0.3 to 0.5 % (bf16's half step)
// after 2^20, 1.5 to 1.8 % after 2^22, as measured.  A longer range of keys is therefore walked in
// pieces of kMostTiles, each from an O of zero and added to the ones before in fp32, rounded to nearest:
// from 2^17 to 2^25 keys an output is off by 0.0019 relative (in one range 0.11 to 0.14 at 2^25), in the
// same time (356 ms for 152 rows of 2^25 keys).
constexpr int kMostTiles = 1024;
// (No wait lasts longer than a piece, about 1.5 ms, however long the sequences are.)
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint64_t kDrainNs = 200000000ull;
constexpr int kSegRing = 4;

enum : int32_t { kWhole, kUncut, kCut };  // how shares take items
// kDirect: the item ends here and its rows can be written; else the state goes to the part `slot`.
// kAgain: another piece of the range came before, whose state is there.
enum : int32_t { kStop = 1, kDirect = 2, kEmpty = 4, kBadLen = 8, kAgain = 16 };

// A share's part of an item, or a piece of it.
struct Segment {
  int32_t row, tokens;    // first packed row, tokens of this tile of rows
  int32_t first, len;     // position of its first token, keys of the sequence
  int32_t b, hk;
  int32_t tile0, tiles;   // key tiles
  int32_t flags, slot;
};

__device__ __forceinline__ bool drain_wait(uint64_t *bar, uint32_t parity) {
  volatile int never = 0;
  return mbar_wait(bar, parity, &never, kDrainNs);
}
__device__ __forceinline__ void fence_async_proxy() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// sum_{i < n} floor((a i + b) / m), a n + b below 2^32, by exchanging the two axes of the lattice
// below the line (Euclid's steps on a and m).
__device__ __forceinline__ int32_t floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  int64_t sum = 0;
#pragma unroll 1
  while (true) {
    if (a >= m) {
      sum += static_cast<int64_t>(n) * (n - 1) / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      sum += static_cast<int64_t>(n) * (b / m);
      b %= m;
    }
    const uint32_t y = a * n + b;
    if (y < m) return static_cast<int32_t>(sum);
    n = y / m;
    b = y % m;
    const uint32_t t = m;
    m = a;
    a = t;
  }
}

// sum_{i < x} floor(i / 2^k)
__device__ __forceinline__ int32_t step_sum(uint32_t x, uint32_t k) {
  const uint32_t q = x >> k, r = x & ((1u << k) - 1);
  return static_cast<int32_t>(((static_cast<uint64_t>(q) * q - q) >> 1 << k) + q * r);
}

// A sequence's new tokens, in tiles of rows, and the steps of these.
struct Seq {
  int32_t row, n, len, first, tiles;  // first: position of its first new token; tiles of rows
  bool bad_len, bad_rows;
  __device__ __forceinline__ Seq() {}
  __device__ __forceinline__ Seq(const RaggedParams &p, int32_t b) {
    row = p.q_start[b];
    const int32_t end = p.q_start[b + 1];
    len = p.kv_len[b];
    bad_rows = row < 0 || end < row || end > p.N;
    n = bad_rows ? 0 : end - row;
    bad_len = len < 0 || len > p.max_pages * p.page_size;
    if (bad_len) len = 0;
    first = len - n;
    tiles = p.by_tokens.div(n + p.tokens - 1);
  }
  // Keys that tile q of rows sees, key tiles (one for a tile that only has rows to write), and the
  // steps of each.
  __device__ __forceinline__ int32_t keys(const RaggedParams &p, int32_t q) const {
    const int32_t last = first + min((q + 1) * p.tokens, n) - 1;
    return last < 0 ? 0 : p.causal ? last + 1 : len;
  }
  __device__ __forceinline__ int32_t units(const RaggedParams &p, int32_t q) const {
    return max(1, (keys(p, q) + kTile - 1) / kTile);
  }
  __device__ __forceinline__ int32_t weight(const RaggedParams &p, int32_t q) const {
    return (n - q * p.tokens) * p.group > kFewRows ? kTileSteps : kFewSteps;
  }
  __device__ __forceinline__ int32_t longest(const RaggedParams &p) const {
    return n > 0 ? kItemSteps + units(p, tiles - 1) * kTileSteps : 0;
  }
  // Steps of tiles 0 .. q - 1 of rows (of all heads: below 2^31, the plan saw to it).
  __device__ __forceinline__ int32_t steps(const RaggedParams &p, int32_t q) const {
    const int32_t whole = min(q, tiles - 1);  // tiles with all their tokens
    int32_t s = 0;
    if (whole > 0) {
      const int32_t idle = first < 0 ? min(whole, p.by_tokens.div(-first)) : 0;
      s = whole;
      if (p.causal) {  // tile i of the others: (first + (i + 1) tokens - 1) / 128 + 1
        if (whole > idle) {
          const uint32_t b = first + (idle + 1) * p.tokens - 1;
          if (p.group_bits >= 0) {  // tokens = 128 / 2^group_bits
            const uint32_t c = b >> (7 - p.group_bits);
            s += step_sum(c + (whole - idle), p.group_bits) - step_sum(c, p.group_bits);
          } else {
            s += floor_sum(whole - idle, kTile, p.tokens, b);
          }
        }
      } else {
        s += (whole - idle) * ((len + kTile - 1) / kTile - 1);
      }
    }
    s = s * kTileSteps + q * kItemSteps;
    if (q > whole) s += units(p, tiles - 1) * weight(p, tiles - 1);
    return s;
  }
};

// Every share's piece of the line: `each` steps, and one more for the first `more`.
struct Line {
  int32_t each, more;
  int32_t mode, shares;
  __device__ __forceinline__ int32_t begin(int32_t share) const {
    return share * each + min(share, more);
  }
  __device__ __forceinline__ int32_t share_of(int32_t step) const {
    const int32_t border = more * (each + 1);
    return step < border ? step / (each + 1) : more + (step - border) / each;
  }
};

// Where a share begins: in sequence b (p.B for nowhere), `left` steps (whole items: items) into it.
struct ShareState {
  unsigned long long rows;
  int32_t total, items, longest, b, left;
  int32_t sums[32];
};

// The sum over the warp of counts whose sum may need more than 32 bits.
__device__ __forceinline__ int64_t warp_count(uint32_t n) {
  return static_cast<int64_t>(__reduce_add_sync(0xffffffffu, n & 0xFFFFu)) +
         (static_cast<int64_t>(__reduce_add_sync(0xffffffffu, n >> 16)) << 16);
}

// How a line of `total` steps in `items` items, the longest of `longest` steps, is shared.
__device__ __forceinline__ Line cut_line(int32_t shares, int32_t total, int32_t items,
                                         int32_t longest) {
  Line line;
  // Whole items, one a share, where the longest is not kJoinSteps longer than equal pieces; where
  // there are more of them than shares, equal pieces with the items that begin in each, at most
  // one longer than equal.
  line.each = total / shares;  // (any number where the rows are wrong: unused then)
  line.mode = items <= shares ? (longest <= line.each + kJoinSteps ? kWhole : kCut)
                              : (longest <= kJoinSteps ? kUncut : kCut);
  line.shares = shares;
  if (line.mode == kCut && line.each < kLeastSteps) {  // a piece holds a tile at least
    line.shares = max(1, total / kLeastSteps);
    line.each = total / line.shares;
  }
  line.more = total - line.each * line.shares;
  return line;
}

__device__ __forceinline__ int32_t steps_of(const RaggedParams &p, const Seq &s) {
  return s.n > 0 ? s.steps(p, s.tiles) * p.kv_heads : 0;
}
__device__ __forceinline__ int32_t warp_scan(int32_t x) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (static_cast<int>(threadIdx.x % 32) >= o) x += y;
  }
  return x;
}

// As many sequences as one warp looks through by itself, two a lane.  More take all of the block's
// threads and some barriers.
constexpr int kFewSequences = 64;

// Finds where share `index` begins, among few sequences (one warp, the result in registers of it
// all).
__device__ __forceinline__ Line find_share_few(const RaggedParams &p, int32_t index, ShareState *st) {
  const int b0 = 2 * (threadIdx.x % 32);
  int32_t steps[2] = {0, 0}, items[2] = {0, 0}, longest = 0;
  int64_t rows = 0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t n = 0;
    if (b0 + k < p.B) {
      const Seq s(p, b0 + k);
      n = s.n;
      steps[k] = steps_of(p, s);
      items[k] = s.tiles * p.kv_heads;
      longest = max(longest, s.longest(p));
      if (s.bad_rows && index == 0) report_bad_page(p.status);
    }
    rows += warp_count(n);
  }
  const Line line = cut_line(p.shares, __reduce_add_sync(0xffffffffu, steps[0] + steps[1]),
                             __reduce_add_sync(0xffffffffu, items[0] + items[1]),
                             __reduce_max_sync(0xffffffffu, longest));
  const bool whole = line.mode == kWhole;
  const int32_t x0 = whole ? items[0] : steps[0], x1 = whole ? items[1] : steps[1];
  const int32_t end = warp_scan(x0 + x1), target = whole ? index : line.begin(index);
  const uint32_t at = __ballot_sync(0xffffffffu, target < end);
  st->b = p.B;
  // (Sequences on top of one another could come to any number of steps: none of them is taken.)
  if (rows > p.N) {
    if (index == 0) report_bad_page(p.status);
    return line;
  }
  if (index < line.shares && at != 0) {
    const int lane = __ffs(at) - 1;
    const int32_t left = target - __shfl_sync(0xffffffffu, end - x0 - x1, lane);
    const int32_t first = __shfl_sync(0xffffffffu, x0, lane);
    st->b = 2 * lane + (left >= first);
    st->left = left >= first ? left - first : left;
  }
  return line;
}

// The same among any number, by all kThreads threads (ends with a barrier; the result in shared
// memory).
template <int kThreads>
__device__ __forceinline__ Line find_share(const RaggedParams &p, int32_t index, ShareState *st) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  if (tid == 0) {
    st->rows = 0;
    st->total = st->items = st->longest = 0;
    st->b = p.B;
  }
  __syncthreads();
  int32_t total = 0, items = 0, mine = 0, mine_items = 0, longest = 0;
  int64_t rows = 0;
  for (int32_t b = tid; b < p.B; b += kThreads) {
    const Seq s(p, b);
    rows += s.n;
    const int32_t t = steps_of(p, s), n = s.tiles * p.kv_heads;
    if (b == tid) {
      mine = t;
      mine_items = n;
    }
    total += t;
    items += n;
    longest = max(longest, s.longest(p));
    if (s.bad_rows && index == 0) report_bad_page(p.status);
  }
  total = __reduce_add_sync(0xffffffffu, total);
  items = __reduce_add_sync(0xffffffffu, items);
  longest = __reduce_max_sync(0xffffffffu, longest);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) rows += __shfl_xor_sync(0xffffffffu, rows, o);
  if (lane == 0 && rows > 0) {
    atomicAdd(&st->rows, static_cast<unsigned long long>(rows));
    atomicAdd(&st->total, total);
    atomicAdd(&st->items, items);
    atomicMax(&st->longest, longest);
  }
  __syncthreads();
  const Line line = cut_line(p.shares, st->total, st->items, st->longest);
  const bool whole = line.mode == kWhole;
  const int32_t target = whole ? index : line.begin(index);
  // (As above.)
  const bool apart = st->rows <= static_cast<unsigned long long>(p.N);
  if (!apart && tid == 0 && index == 0) report_bad_page(p.status);
  const int32_t all = whole ? st->items : st->total;
  if (apart && index < line.shares && target < all) {  // uniform
    int32_t base = 0;
    for (int32_t b0 = 0; b0 < p.B && base <= target; b0 += kThreads) {
      int32_t x = 0;
      if (b0 == 0) {
        x = whole ? mine_items : mine;
      } else if (b0 + tid < p.B) {
        const Seq s(p, b0 + tid);
        x = whole ? s.tiles * p.kv_heads : steps_of(p, s);
      }
      const int32_t incl = warp_scan(x);
      if (lane == 31) st->sums[warp] = incl;
      __syncthreads();
      int32_t before = base, chunk = 0;
      for (int w = 0; w < kThreads / 32; ++w) {
        const int32_t y = st->sums[w];
        chunk += y;
        if (w < warp) before += y;
      }
      before += incl - x;
      if (before <= target && target < before + x) {
        st->b = b0 + tid;
        st->left = target - before;
      }
      base += chunk;
      __syncthreads();
    }
  }
  __syncthreads();
  return line;
}

// A share's walk along its items (one warp, uniform).
struct Walk {
  Seq s;
  int32_t b, hk, q, units, weight;
  int32_t tile;  // the next key tile of the item
  int32_t end;   // the share's end, in steps from the item's first tile
  bool cut;
  __device__ __forceinline__ Walk(const RaggedParams &p, const Line &line, int32_t index,
                                  const ShareState &st)
      : b(st.b), hk(0), q(0), units(1), weight(1), tile(0), end(-kItemSteps),
        cut(line.mode == kCut) {
    if (b >= p.B) return;
    s = Seq(p, b);
    int32_t rest = st.left;
    if (line.mode == kWhole) {
      hk = rest / s.tiles;
      q = rest - hk * s.tiles;
      item(p);
      end = units * weight;
      return;
    }
    const int32_t head = s.steps(p, s.tiles);
    hk = rest / head;
    rest -= hk * head;
    // The last tile of rows whose steps begin at or before `rest`, 32 candidates at a time.
    int32_t lo = 0, hi = s.tiles;
    while (hi - lo > 1) {
      const int32_t step = (hi - lo + 31) / 32, x = lo + static_cast<int32_t>(threadIdx.x % 32) * step;
      const bool before = x < hi && s.steps(p, x) <= rest;
      const int top = 31 - __clz(__ballot_sync(0xffffffffu, before));
      lo += top * step;
      hi = min(hi, lo + step);
    }
    q = lo;
    item(p);
    const int32_t off = rest - s.steps(p, q) - kItemSteps;  // of the share's begin from the tiles
    end = off + line.each + (index < line.more ? 1 : 0);
    if (cut) {
      tile = off > 0 ? (off + weight - 1) / weight : 0;
      if (tile == units) next(p);
    } else if (off > -kItemSteps) {
      next(p);
    } else {
      take_whole();
    }
  }
  __device__ __forceinline__ bool more(const RaggedParams &p) const {
    return b < p.B && tile * weight < end;
  }
  // The share's part of the item.
  __device__ __forceinline__ Segment segment(const RaggedParams &p, int32_t share) const {
    const int32_t t0 = q * p.tokens;
    Segment g;
    g.row = s.row + t0;
    g.tokens = min(p.tokens, s.n - t0);
    g.first = s.first + t0;
    g.len = s.len;
    g.b = b;
    g.hk = hk;
    g.tile0 = tile;
    g.tiles = (end > (units - 1) * weight ? units : (end + weight - 1) / weight) - tile;
    g.flags = (g.tiles == units ? kDirect : 0) | (s.keys(p, q) == 0 ? kEmpty : 0) |
              (s.bad_len ? kBadLen : 0);
    g.slot = 2 * share + (tile == 0 ? 1 : 0);
    return g;
  }
  // Of a cut item that begins in the share.
  __device__ __forceinline__ RaggedJoin join(const Line &line, int32_t share, const Segment &g) const {
    const int32_t last = line.begin(share + 1) - end + (units - 1) * weight;  // its last tile's place
    return {line.share_of(last) - share + 1, g.slot, g.hk, g.row, g.tokens, g.first, {0, 0}};
  }
  __device__ __forceinline__ void item(const RaggedParams &p) {
    units = s.units(p, q);
    weight = s.weight(p, q);
  }
  // Uncut: the items that begin in the share are all its own.
  __device__ __forceinline__ void take_whole() {
    if (!cut && end > -kItemSteps) end = max(end, units * weight);
  }
  __device__ __forceinline__ void next(const RaggedParams &p) {
    end -= units * weight + kItemSteps;
    tile = 0;
    if (++q == s.tiles) {
      q = 0;
      if (++hk == p.kv_heads) {
        hk = 0;
        // (In cut lines an item whose first tile is past the end has no part here.)
        do {
          if (++b == p.B || end <= (cut ? 0 : -kItemSteps)) return;
          s = Seq(p, b);
        } while (s.n == 0);
      }
    }
    item(p);
    take_whole();
  }
};

// The next piece of a share's part of an item, of whose tiles `rest` are left.
__device__ __forceinline__ Segment piece_of(Segment g, int32_t rest) {
  if (rest < g.tiles) g.flags |= kAgain;
  if (rest > kMostTiles) g.flags &= ~kDirect;
  g.tile0 += g.tiles - rest;
  g.tiles = min(kMostTiles, rest);
  return g;
}

// Two states of a row over different keys: the common reference, the sum, and what either's O counts
// times.
struct Merge {
  float m, l, before, now;
};
__device__ __forceinline__ Merge merge_states(float m0, float l0, float m1, float l1) {
  Merge x;
  x.m = fmaxf(m0, m1);
  x.before = m0 == x.m ? 1.f : exp2f(m0 - x.m);
  x.now = m1 == x.m ? 1.f : exp2f(m1 - x.m);
  x.l = l0 * x.before + l1 * x.now;
  return x;
}

// Where a key warp or a value warp is in its ring.
template <int kSlots>
struct Ring {
  uint32_t n = 0;  // uses so far
  __device__ __forceinline__ int slot() const { return n % kSlots; }
  __device__ __forceinline__ bool wait_empty(uint64_t *empty, volatile int *abort) const {
    return n < kSlots ||
           mbar_wait_warp(&empty[slot()], ((n - kSlots) / kSlots) & 1, abort, kWaitNs);
  }
  __device__ __forceinline__ void drain(uint64_t *full) const {  // of the copies still in flight
    for (uint32_t c = n > kSlots ? n - kSlots : 0; c < n; ++c)
      drain_wait(&full[c % kSlots], (c / kSlots) & 1);
  }
};

// The key of a tile from which on some row of the segment does not see it, or there is none.
__device__ __forceinline__ int32_t seen_by_all(const RaggedParams &p, const Segment &g) {
  return p.causal ? min(max(g.first, 0), g.len - 1) : g.len - 1;
}

// Values that not all rows see must not reach the others through a zero weight (0 * inf is not
// zero): of a tile's keys past `seen` those behind the sequence's end become zero, and values of the
// others that are not finite as well, in shared memory, before the tile's product.  The softmax
// warps do this, 16 rows each, once they have the tile's weights: one warp beside them took 2.2 us
// (d = 64) and 3 us for a tile, in which the tensor cores waited at each item's end.
//
// Zero times a value is zero, or NaN where the value is not finite, and so is a sum of such: one
// instruction looks at two values.  (Keys that all rows see may count too; fix_each tells them
// apart.)  True where the warp's rows hold one.
template <int kBlocks>
__device__ __forceinline__ bool fix_rows(uint8_t *tile, int32_t row0, int32_t key0, int32_t seen,
                                         int32_t len) {
  if (key0 + row0 + 15 <= seen) return false;
  const int lane = threadIdx.x % 32;
  const int end = len - key0;  // rows of the sequence
  const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
  __nv_bfloat162 odd[4] = {zero, zero, zero, zero};
#pragma unroll
  for (int k0 = 0; k0 < kBlocks; k0 += 2) {
    uint4 x[4][2];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = row0 + 4 * j + (lane >> 3);
        uint4 *at = reinterpret_cast<uint4 *>(tile + (k0 + k) * (kTile * 128) + row * 128 +
                                              ((lane & 7) << 4));
        x[j][k] = make_uint4(0, 0, 0, 0);
        if (row < end)
          x[j][k] = *at;
        else
          *at = x[j][k];
      }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const __nv_bfloat162 *v = reinterpret_cast<const __nv_bfloat162 *>(&x[j][k]);
#pragma unroll
        for (int i = 0; i < 4; ++i) odd[i] = __hfma2(v[i], zero, odd[i]);
      }
  }
  const __nv_bfloat162 any = __hadd2(__hadd2(odd[0], odd[1]), __hadd2(odd[2], odd[3]));
  return __any_sync(0xffffffffu, __hisnan(any.x) || __hisnan(any.y));
}

// Such rows: each value past `seen` that is not finite becomes zero, and its column's byte the
// least distance from `seen` of such a key (at most 254; 255 where there is none): rows at least
// that far from `seen` see it.  Broken models' values only, so short rather than fast.
template <int kBlocks>
__device__ __noinline__ void fix_each(uint8_t *tile, int32_t row0, int32_t key0, int32_t seen,
                                      int32_t len, uint32_t *columns) {
  const int lane = threadIdx.x % 32;
  for (int x = lane; x < 16 * kBlocks * 32; x += 32) {  // words of two columns
    const int row = row0 + x / (kBlocks * 32), word = x % (kBlocks * 32);
    const int32_t far = key0 + row - seen;
    if (far <= 0 || key0 + row >= len) continue;
    const int chunk = word % 32 / 4;
    uint32_t *at = reinterpret_cast<uint32_t *>(tile + word / 32 * (kTile * 128) + row * 128 +
                                                ((chunk ^ (row & 7)) << 4)) + word % 4;
    const uint32_t w = *at;
    const bool lo = (w & 0x7F80u) == 0x7F80u, hi = (w & 0x7F800000u) == 0x7F800000u;
    if (!lo && !hi) continue;
    *at = w & ((lo ? 0xFFFF0000u : 0xFFFFFFFFu) & (hi ? 0xFFFFu : 0xFFFFFFFFu));
    const uint32_t d = min(254, far);
    const uint32_t two = (lo ? d : 255u) | ((hi ? d : 255u) << 8);
    const uint32_t mine = word % 2 ? (two << 16) | 0xFFFFu : two | 0xFFFF0000u;
    uint32_t old = columns[word / 2], now;
    while ((now = __vminu4(old, mine)) != old) {
      const uint32_t was = atomicCAS(&columns[word / 2], old, now);
      if (was == old) break;
      old = was;
    }
  }
  __syncwarp();
}

// The first warp that needs a segment's column bytes (there are two sets, in turn) sets them to 255
// once the segment before last has been read; `state` goes from 0 over 1 to 2.  False where a wait
// ran out.
__device__ __noinline__ bool open_columns(int32_t *state, uint32_t *columns, int words,
                                          uint64_t *before_last, uint32_t parity, bool any_before,
                                          volatile int *abort) {
  const int lane = threadIdx.x % 32;
  int32_t was = 0;
  if (lane == 0) was = atomicCAS(state, 0, 1);
  was = __shfl_sync(0xffffffffu, was, 0);
  if (was == 0) {
    if (any_before && !mbar_wait_warp(before_last, parity, abort, kWaitNs)) return false;
    for (int x = lane; x < words; x += 32) columns[x] = 0xFFFFFFFFu;
    __threadfence_block();
    __syncwarp();
    if (lane == 0) atomicExch(state, 2);
    return true;
  }
  const uint64_t t0 = globaltimer_ns();
  while (*reinterpret_cast<volatile int32_t *>(state) != 2) {
    if (globaltimer_ns() - t0 > kWaitNs) *abort = 1;
    if (*abort) return false;
  }
  __threadfence_block();
  return true;
}

// The page of the piece of a tile that begins at `key` of sequence b.  (Each kernel has a warp that
// loads keys, walks along the share and describes its segments, and one that loads values.  A tile is
// pieces of piece_rows rows, each in one page, in boxes 128 bytes wide, a copy and a lane each: lane =
// piece * boxes + box.)
__device__ __forceinline__ int32_t page_of(const RaggedParams &p, int32_t b, int32_t len, int32_t key,
                                           bool piece_ok) {
  return piece_ok && key < len
             ? p.page_table[static_cast<int64_t>(b) * p.max_pages + p.by_page.div(key)]
             : 0;
}

}  // namespace
}  // namespace diffattn
