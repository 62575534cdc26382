// diffpaged_evict: cut a paged cache down to the keys of the largest
// accumulated weights.
//
// Per (sequence, key/value head) with len > keep keys: the last `recent` stay,
// and of the first old = len - recent the k = keep - recent largest weights,
// the lower position first among equals.  The kept rows move to positions
// 0 .. keep - 1 in their order, in place.
//
//   1. Select (one block per item).  Weights become 32-bit keys whose unsigned
//      order is theirs (sign flipped or all bits; NaN as +infinity, -0 as 0);
//      three histogram passes over 11 + 11 + 10 bits find the k-th largest
//      value T and how many equal to T still fit; a scan in position order
//      then writes the list of kept places and moves the weights.  A thread
//      holds up to 16 consecutive weights in registers, so up to 16384 keys
//      are read once and ordered by one scan; longer sequences take more
//      rounds over a copy.
//   2. Move (one block per item and 128-byte column slice of k1, k2, v).  A
//      kept row's place is at or before its source, and sources ascend, so
//      blocks of rows taken in order only need all loads of a block before
//      its stores; the slices are independent of one another.  The next
//      rows' places are fetched while a block of rows is on its way.
//
// Bound: HBM, each kept row read and written once.
#include <cuda_runtime.h>

#include <cstdint>

#include "debug_check.cuh"
#include "paged.h"
#include "ptx.cuh"

namespace diffattn {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int kBatch = 4;   // 16-byte units of a thread in a block of rows
constexpr int kAhead = 3;   // blocks of rows in flight
constexpr int kHeld = 16;   // weights that a thread of the selection holds

struct EvictParams {
  uint8_t *pool[3];
  int64_t page_b[3], head_b[3], row_b[3];  // strides in bytes
  int32_t width_b[3];                      // bytes of a row
  float *weights;
  const int32_t *page_table;
  int32_t *kv_len;
  int32_t *status;
  int32_t B, kv_heads, num_pages, max_pages, page_size;
  int32_t keep, recent;
  FastDiv by_page;
  int64_t padded;   // entries per item of copy
  float *copy;      // [items][padded] the item's weights by position, where they take rounds
  int2 *list;       // [items][keep] page and slot of each kept row
  int2 *plan;       // [items] {rows already in place, 1}; {0, 0}: nothing to do
};

__device__ __forceinline__ uint32_t order_key(float w) {
  if (isnan(w)) w = INFINITY;
  const uint32_t x = __float_as_uint(w + 0.f);  // -0 becomes 0
  return (x & 0x80000000u) ? ~x : x | 0x80000000u;
}

// Exclusive prefix sum over the block; *total gets the whole sum.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t *scratch, uint32_t *total) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  uint32_t incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    uint32_t s = scratch[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    scratch[lane] = s;
  }
  __syncthreads();
  const uint32_t before = warp == 0 ? 0 : scratch[warp - 1];
  *total = scratch[31];
  __syncthreads();
  return before + incl - x;
}

__device__ __forceinline__ bool in_order(uint32_t key, uint32_t prefix, int shift) {
  return shift >= 32 || key >> shift == prefix >> shift;
}

__global__ void __launch_bounds__(kSelectThreads) diffpaged_select_kernel(const EvictParams p) {
  __shared__ uint32_t hist[2048];
  __shared__ uint32_t scratch[32];
  __shared__ uint32_t found[2];
  const int item = blockIdx.x, tid = threadIdx.x;
  const int b = item / p.kv_heads, hk = item % p.kv_heads;
  for (int i = tid; i < 2048; i += kSelectThreads) hist[i] = 0;
  grid_dependency_wait();
  grid_dependents_launch();
  const int32_t len = __ldg(p.kv_len + b);
  const bool bad_len = len < 0 || len > p.max_pages * p.page_size;
  if (bad_len || len <= p.keep) {
    if (tid == 0) {
      if (bad_len) report_bad_page(p.status);
      p.plan[item] = make_int2(0, 0);
    }
    return;
  }
  const int32_t *table = p.page_table + static_cast<int64_t>(b) * p.max_pages;
  const int32_t old = len - p.recent;
  const uint32_t k_keep = p.keep - p.recent;
  float *copy = p.copy + item * p.padded;
  const auto weights_of = [&](int32_t page) {
    return p.weights + (static_cast<int64_t>(page) * p.kv_heads + hk) * p.page_size;
  };

  // Rounds of 1024 threads x `each` consecutive positions, in groups of four (which no page
  // boundary cuts); one round up to 16384 positions.
  const int32_t each = min(kHeld, ((len + kSelectThreads - 1) / kSelectThreads + 3) & ~3);
  const int32_t per_round = each * kSelectThreads;
  const bool single = len <= per_round;
  float w[kHeld];
  bool bad = false;
  const auto load = [&](int32_t at, bool first) {  // this thread's weights of the round at `at`
    const int32_t j0 = at + tid * each;
#pragma unroll
    for (int g = 0; g < kHeld; g += 4) {
      if (g >= each || j0 + g >= len) break;
      const float *src = copy + j0 + g;
      if (first) {
        const int32_t n = p.by_page.div(j0 + g);
        const int32_t page = __ldg(table + n);
        bad |= static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.num_pages);
        if (bad) break;
        src = weights_of(page) + (j0 + g - n * p.page_size);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (j0 + g + e < len) w[g + e] = src[e];
    }
  };

  // The k-th largest key, from its leading bits down.
  uint32_t prefix = 0, need = k_keep;  // need: how many are still to be found at or below prefix
  const int shift[3] = {21, 10, 0}, bits[3] = {11, 11, 10};
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    for (int32_t at = 0; at < len; at += per_round) {
      if (pass == 0 || !single) load(at, pass == 0);
      const int32_t j0 = at + tid * each;
#pragma unroll
      for (int g = 0; g < kHeld; ++g) {
        if (g >= each) break;
        const int32_t j = j0 + g;
        if (pass == 0 && !single && j < len) copy[j] = w[g];
        const uint32_t key = order_key(w[g]);
        const bool counts = j < old && in_order(key, prefix, shift[pass] + bits[pass]);
        const uint32_t bin = counts ? (key >> shift[pass]) & ((1u << bits[pass]) - 1) : 0xFFFFFFFFu;
        // Equal weights fill one bin: a warp that agrees adds once.
        int same;
        __match_all_sync(0xffffffffu, bin, &same);
        if (same) {
          if (counts && tid % 32 == 0) atomicAdd(&hist[bin], 32u);
        } else if (counts) {
          atomicAdd(&hist[bin], 1u);
        }
      }
    }
    if (__syncthreads_or(bad)) {  // a page of the sequence is not one: it stays as it is
      if (tid == 0) {
        report_bad_page(p.status);
        p.plan[item] = make_int2(0, 0);
      }
      return;
    }
    // Thread t holds bins 2047 - 2 t and 2046 - 2 t: sums from the largest bin down.
    const uint32_t hi = hist[2047 - 2 * tid], lo = hist[2046 - 2 * tid];
    hist[2047 - 2 * tid] = hist[2046 - 2 * tid] = 0;
    if (tid == 0) found[0] = found[1] = 0;
    uint32_t total;
    const uint32_t above = block_scan(hi + lo, scratch, &total);
    if (need > above && need <= above + hi + lo) {
      const bool in_hi = need <= above + hi;
      found[0] = in_hi ? 2047 - 2 * tid : 2046 - 2 * tid;
      found[1] = need - above - (in_hi ? 0 : hi);
    }
    __syncthreads();
    prefix |= found[0] << shift[pass];
    need = found[1];
  }

  // Kept places in order: keys above T, the first `need` equal to it, and the last `recent`.
  uint32_t equal_before = 0, kept = 0;
  int2 *list = p.list + static_cast<int64_t>(item) * p.keep;
  uint32_t in_place = 0xFFFFFFFFu;  // the first position that does not stay
  for (int32_t at = 0; at < len; at += per_round) {
    if (!single) load(at, false);
    const int32_t j0 = at + tid * each;
    uint32_t equal = 0, all_equal = 0;
#pragma unroll
    for (int g = 0; g < kHeld; ++g)
      if (g < each && j0 + g < old) equal += order_key(w[g]) == prefix ? 1 : 0;
    uint32_t eq = equal_before + block_scan(equal, scratch, &all_equal);
    uint32_t mask = 0;
#pragma unroll
    for (int g = 0; g < kHeld; ++g) {
      const int32_t j = j0 + g;
      if (g >= each || j >= len) break;
      const uint32_t key = order_key(w[g]);
      const bool is_equal = key == prefix;
      const bool stays = j >= old || (k_keep > 0 && (key > prefix || (is_equal && eq < need)));
      if (j < old && is_equal) ++eq;
      if (stays)
        mask |= 1u << g;
      else
        in_place = min(in_place, static_cast<uint32_t>(j));
    }
    uint32_t total;
    uint32_t to = kept + block_scan(__popc(mask), scratch, &total);
    // Every weight of this round has been read (and, in more rounds, of all: from the copy).
#pragma unroll
    for (int g = 0; g < kHeld; ++g) {
      if (!((mask >> g) & 1) || !dbg_ok(to < static_cast<uint32_t>(p.keep), p.status, 50)) continue;
      const int32_t n = p.by_page.div(j0 + g), m = p.by_page.div(static_cast<int32_t>(to));
      list[to] = make_int2(__ldg(table + n), j0 + g - n * p.page_size);
      weights_of(__ldg(table + m))[to - m * p.page_size] = w[g];
      ++to;
    }
    equal_before += all_equal;
    kept += total;
  }
  in_place = __reduce_min_sync(0xffffffffu, in_place);
  if (tid % 32 == 0) scratch[tid / 32] = in_place;
  __syncthreads();
  if (tid < 32) {
    in_place = __reduce_min_sync(0xffffffffu, scratch[tid]);
    if (tid == 0) p.plan[item] = make_int2(min(static_cast<int32_t>(in_place), p.keep), 1);
  }
}

__global__ void __launch_bounds__(kMoveThreads) diffpaged_move_kernel(const EvictParams p,
                                                                      int slices) {
  const int item = blockIdx.x / slices;
  int slice = blockIdx.x - item * slices;
  const int b = item / p.kv_heads, hk = item - b * p.kv_heads;
  int t = 0;
  while (slice >= (p.width_b[t] + 127) / 128) slice -= (p.width_b[t++] + 127) / 128;
  const int units = p.width_b[t] < 128 ? p.width_b[t] / 16 : 8;  // 16-byte units of the slice
  const int unit = threadIdx.x & (units - 1), line = threadIdx.x / units;
  const int lines = kMoveThreads / units;  // rows taken side by side
  uint8_t *base = p.pool[t] + hk * p.head_b[t] + slice * 128 + unit * 16;
  const int64_t page_b = p.page_b[t], row_b = p.row_b[t];
  const int32_t *table = p.page_table + static_cast<int64_t>(b) * p.max_pages;
  const int2 *list = p.list + static_cast<int64_t>(item) * p.keep;
  grid_dependency_wait();
  grid_dependents_launch();
  const int2 plan = p.plan[item];
  if (plan.y == 0) return;
  if (blockIdx.x == b * p.kv_heads * slices && threadIdx.x == 0) p.kv_len[b] = p.keep;
  // A ring of row blocks in shared memory.  A thread stores what it loaded itself; the barrier
  // makes every source of a block be read before any of its places is written, and the sources of
  // the blocks after lie behind those places.
  __shared__ uint4 ring[kAhead][kBatch][kMoveThreads];
  int2 from[kBatch];  // places of the next block's rows
  const auto look_up = [&](int32_t first) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int32_t at = first + u * lines + line;
      if (at < p.keep) from[u] = list[at];
    }
  };
  const auto fetch = [&](int32_t first, int stage) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (first + u * lines + line < p.keep)
        cp_async16(smem_u32(&ring[stage][u][threadIdx.x]),
                   base + from[u].x * page_b + from[u].y * row_b);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const int32_t step = lines * kBatch;
  int32_t ahead = plan.x;
  look_up(ahead);
#pragma unroll
  for (int k = 0; k < kAhead - 1; ++k) {
    fetch(ahead, k);
    ahead += step;
    look_up(ahead);
  }
  int stage = 0;
#pragma unroll 1
  for (int32_t first = plan.x; first < p.keep; first += step) {
    fetch(ahead, (stage + kAhead - 1) % kAhead);
    ahead += step;
    look_up(ahead);
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int32_t at = first + u * lines + line;
      if (at < p.keep) {
        const int32_t n = p.by_page.div(at);
        *reinterpret_cast<uint4 *>(base + __ldg(table + n) * page_b +
                                   (at - n * p.page_size) * row_b) = ring[stage][u][threadIdx.x];
      }
    }
    stage = (stage + 1) % kAhead;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

struct EvictLayout {
  size_t copy, list, plan, bytes;
  int64_t padded;
};

EvictLayout layout(const diffattn_desc &desc, const diffpaged_cache &cache, int64_t keep) {
  EvictLayout l;
  const int64_t items = desc.B * cache.kv_heads;
  const int64_t most = cache.max_pages * cache.page_size;
  l.padded = most;
  const int64_t kept = keep < most ? keep : most;
  l.copy = 0;
  const int64_t copied = most > kHeld * kSelectThreads ? most : 0;
  l.list = round256(static_cast<size_t>(items * copied) * sizeof(float));
  l.plan = l.list + round256(static_cast<size_t>(items * kept) * sizeof(int2));
  l.bytes = l.plan + round256(static_cast<size_t>(items) * sizeof(int2));
  return l;
}

}  // namespace

size_t paged_evict_bytes(const diffattn_desc &desc, const diffpaged_cache &cache, int64_t keep) {
  // A budget that no sequence can pass needs nothing.
  if (keep >= cache.max_pages * cache.page_size || desc.B == 0) return 0;
  return layout(desc, cache, keep).bytes;
}

diffattn_status launch_paged_evict(const diffattn_desc &desc, const diffpaged_cache &cache,
                                   int64_t keep, int64_t recent, void *workspace,
                                   cudaStream_t stream) {
  if (keep >= cache.max_pages * cache.page_size) return DIFFATTN_OK;
  const bool fp8 = desc.dtype == DIFFATTN_E4M3_QK;
  const EvictLayout l = layout(desc, cache, keep);
  EvictParams p = {};
  void *pool[3] = {cache.k1, cache.k2, cache.v};
  const diffattn_strides *st[3] = {&cache.k1_strides, &cache.k2_strides, &cache.v_strides};
  int slices = 0;
  for (int t = 0; t < 3; ++t) {
    const int64_t es = fp8 && t < 2 ? 1 : 2;
    p.pool[t] = static_cast<uint8_t *>(pool[t]);
    p.page_b[t] = es * st[t]->b;
    p.head_b[t] = es * st[t]->h;
    p.row_b[t] = es * st[t]->n;
    p.width_b[t] = static_cast<int32_t>(es * (t == 2 ? 2 * desc.d : desc.d));
    slices += (p.width_b[t] + 127) / 128;
  }
  p.weights = cache.weights;
  p.page_table = cache.page_table;
  p.kv_len = cache.kv_len;
  p.status = desc.status_dev;
  p.B = static_cast<int32_t>(desc.B);
  p.kv_heads = static_cast<int32_t>(cache.kv_heads);
  p.num_pages = static_cast<int32_t>(cache.num_pages);
  p.max_pages = static_cast<int32_t>(cache.max_pages);
  p.page_size = cache.page_size;
  p.keep = static_cast<int32_t>(keep);
  p.recent = static_cast<int32_t>(recent);
  p.by_page = fast_div(static_cast<uint32_t>(p.page_size));
  p.padded = l.padded;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  p.copy = reinterpret_cast<float *>(ws + l.copy);
  p.list = reinterpret_cast<int2 *>(ws + l.list);
  p.plan = reinterpret_cast<int2 *>(ws + l.plan);
  const double items = static_cast<double>(desc.B) * static_cast<double>(cache.kv_heads);
  if (items * slices > INT32_MAX) return DIFFATTN_ERR_UNSUPPORTED;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items));
  cfg.blockDim = dim3(kSelectThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, diffpaged_select_kernel, p) != cudaSuccess) return DIFFATTN_ERR_CUDA;
  cfg.gridDim = dim3(static_cast<unsigned>(items) * slices);
  cfg.blockDim = dim3(kMoveThreads);
  return cudaLaunchKernelEx(&cfg, diffpaged_move_kernel, p, slices) == cudaSuccess
             ? DIFFATTN_OK
             : DIFFATTN_ERR_CUDA;
}

}  // namespace diffattn
