// diffpaged_fwd: the differential head's forward of a few new tokens per
// sequence over a paged key/value cache.
//
// The mathematics.  The rows of one (sequence, key/value head) are r = (token
// i, query head g of the group), R = N * G of them, all reading the same keys:
//   x_m[r, j] = q_m[r] . k_m[j] / sqrt(d),  map_m = softmax_j(x_m),  m = 1, 2
//   o[r] = sum_j (map1[r, j] - lambda_h map2[r, j]) v[j], then the head norm.
// Each map is an ordinary softmax, so the keys are taken in one pass with a
// running reference maximum and sum per row and map (fp32, log2 units), and
// ranges of keys done by different CTAs join exactly: with M = max m_s,
//   O = sum_s 2^(m_s - M) O_s,  l = sum_s 2^(m_s - M) l_s,  o = O / l.
//
// What bounds it: each key is read once (8 d bytes in bf16) for 12 d R
// multiply-adds, so for the R <= 32 rows of a block this is HBM-bound, and
// everything here serves to keep loads in flight.
//
//   - Work is counted in tiles of 128 keys over all sequences and heads, and
//     every CTA (one per SM) takes the same share of consecutive tiles, found
//     from kv_len on the device; a ragged batch is balanced and a graph
//     replays with new lengths.  Items cut by a CTA boundary leave partial
//     states, which a second kernel (launched dependent on the first) joins.
//     Where the lengths make that longer by a few tiles only (few tiles in all,
//     many short items), one CTA takes each item, or each the items that begin
//     in its share, and nothing is joined.  Both kernels choose alike from the
//     lengths (18 x 8 heads of 100 to 9001 keys, 144 items for 152 SMs: chosen
//     from the capacity of the page table 74 us, from the lengths 60 us; 19 x 8
//     with one sequence of 32768 keys beside others of 200: 236 and 33 us).
//   - Two warps issue TMA copies of page pieces (16 to 64 rows, by the page
//     size), one of keys and one of values, into rings of 32 KB buffers, 128 to
//     192 KB in all: the keys of both maps (d = 64 or e4m3), one map's keys or
//     128 value columns.  The copies leave L2 first (evict_first): a cache is
//     read once a step, and without the hint it pushes out even the kernel's
//     code (8 x 8K keys: 55 -> 51 us).  A third warp fetches the q rows.
//   - One warp issues the products, keys and value columns on the 128-row side
//     of tcgen05.mma, where the tile fills it, and the few rows r on the other:
//       S_m^T = K_m Q_m^T            (128 keys x rows)
//       O^T  += V^T [P1 | P2]^T      (128 value columns x rows of both maps)
//     so V is read once for both maps and O stays in tensor memory.
//   - Eight warps (16 from 8 rows on) do the softmax, a thread per key and map.
//     The reference maximum moves only when some logit passes it by 2^8: one
//     barrier with a vote per tile instead of a reduction over the keys.
//   - The end of a segment (a CTA's part of an item) is done after the next
//     tile's softmax, so that its last product runs meanwhile.  Its code and
//     that of the first tile run once or a few times a call, so they are kept
//     short: fetching them costs more than executing them (three tiles of 20
//     rows, with each row's sums reduced in turn and inlined: 18.9 us, with
//     all rows in one exchange: 14.4 us).
//   - P enters the second product as bf16 hi + lo side by side (relative
//     error 2^-17): o1 - lambda o2 cancels and the head norm scales the
//     difference back up, so a plain bf16 P would show; the wider product is
//     hidden behind the loads.
//
// Measured on GB300 (device time of a call, join included; the copy rate is
// 6.78 TB/s): 32 heads x 16384 keys in pages of 64, 268 MB: 47 us, 84 % of it;
// 8 sequences x 8 heads x 8192 keys at d = 128, 537 MB: 84 us, 94 %; 24
// sequences of 100 to 9001 keys in pages of 16, four query heads to a key/value
// head, 448 MB: 76 us, 87 %; 8 x 8 x 32768 keys, 1.07 GB: 163 to 167 us, 95 to
// 97 %; one sequence of 200 keys, 16 heads: 6.3 us, of which 2.5 us pass before
// the first copy lands.  Of a large call's time beyond the copy rate about 3 us
// go to the first lookups and copies and 3 us to the join; with 32 rows the
// softmax bounds it (8 x 8K keys: 16 rows 53 us, 32 rows 78 to 83 us).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "debug_check.cuh"
#include "paged.h"
#include "ptx.cuh"

namespace diffattn {

struct FwdParams {
  const void *q1, *q2;
  const void *v_pages;
  const float *lambda, *norm_w;
  __nv_bfloat16 *out;
  const int32_t *page_table, *kv_len;
  int32_t *status;
  diffattn_strides q1s, q2s, outs, vs;
  int32_t B, H, N, kv_heads, group, rows;  // rows = N * group
  int32_t num_pages, max_pages, page_size, piece_rows;
  int32_t row_blocks, causal, headnorm;
  int32_t mode;  // PagedMode
  FastDiv by_page, by_group;  // page_size, group
  float eps, out_scale, scale_log2;
  // Workspace (see PagedFwdPlan): partial O [2 C][2][NR][2 d] and their (m, l), and for accumulate
  // whole items' (m, l) and all logits.
  float *part;
  float2 *part_ml;
  float2 *item_ml;
  // [B * kv_heads][2][planes][padded][rows of a plane], log2 units, or null: the rows in planes of
  // (up to) four, so that a thread stores those of its key at once and a warp whole lines.
  float *logits;
  int64_t padded;
  int32_t planes;
  float *weights;
};

namespace {

constexpr int kTile = kPagedTile;
// Warps 0-2 issue, those from 4 on (a multiple of four, for their quarters of tensor memory) do the
// softmax.
constexpr int kMmaWarp = 0, kKeyWarp = 1, kValueWarp = 2, kQueryWarp = 3, kSoftmaxWarp = 4;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint64_t kDrainNs = 200000000ull;
constexpr float kGrowth = 8.f;  // log2 units a logit may pass the reference maximum by
// A reference before any key above -infinity is seen: finite, so that such a key's 2^(x - m) is 0.
constexpr float kLeast = -FLT_MAX;
constexpr int kMaxBad = 16;     // as many as new tokens: more than keys that only some of them see
constexpr int kRing = 8;        // tile descriptors; fewer tiles are between load and epilogue
constexpr int kBoxBytes = kTile * 128;   // 64 bf16 columns of a tile
constexpr int kSlotBytes = 2 * kBoxBytes;
constexpr int kItemCost = 2;    // steps, see Shares
// One CTA per item, and nothing to join, where equal shares would not save this many tiles of the
// longest, what the join and the second segment of most CTAs take (6 us, of 1 us a tile).  64 items
// of 8 tiles on 152 SMs: 12.0 us, cut 14.1; of 16 tiles 18.6 and 18.4; 16 items of 4 tiles 7.7 and
// 8.3, of 8 tiles 10.8 and 9.6; 128 items of 500 to 1500 keys 18.0 and 19.3; 64 of 100 to 1500 keys
// (cut: it would be 9.2 tiles) 15.0 and 13.8.
constexpr int kMostAlone = 6;
// What a second kernel takes that finds nothing to do (64 x 16 heads of 200 keys: 24.8 us, and 26.3
// under a table of 4096 keys, which other lengths could have cut).
constexpr int kSecondKernel = 2;
// Nor are items cut where they are so many, or so short, that no share gets this many steps longer
// by taking them whole, which costs less than the join.  408 items of two tiles (8 rows): 18.5 us,
// cut 22.4; 1024 of two: 24.8 and 27.8; 228 of six (32 rows, d = 128): 54 and 63; 240 of ten, where
// it would be 5.05 steps: 30.5 and 31.5; 456 of 500 to 900 keys, where it could be more: 33.2 and
// 33.6.
constexpr int kUneven = 5;
constexpr float kLog2e = 1.4426950408889634f;

enum : int32_t { kFirst = 1, kLast = 2, kStop = 4, kBad = 8, kDirect = 16 };

struct TileDesc {
  int32_t b, hk, real, key0;  // real: rows of the block
  int32_t len, flags, slot, item;
  int32_t steps;  // 16-key steps of the second product (one for an idle sequence)
  int32_t rb, pad[2];
};


// One row of a segment, as the softmax warps need it.
struct RowInfo {
  int32_t last;   // the last key that it sees, -1 for none
  int32_t head;   // query head
  int64_t out;    // element offset of its output
};

// kNR: rows of a block (1, 2, 4, 8, 16 or 32), padded to kNQ = 8, 16 or 32 in the products.
template <int kD, bool kFp8, int kNR>
struct Geo {
  static constexpr int kNQ = kNR < 8 ? 8 : kNR;
  // Softmax threads: one per key and map, two from 8 rows on, with half of the rows each.
  static constexpr int kSets = kNR < 8 ? 1 : 2;
  static constexpr int kConsumers = 2 * kTile * kSets;
  static constexpr int kThreads = 32 * kSoftmaxWarp + kConsumers;
  static constexpr int kMine = kNR / kSets;                         // rows of a thread
  static constexpr int kW = kMine < 8 ? kMine : 8;                  // of them at a time
  static constexpr int kChunks = kMine / kW;
  static constexpr int kKeyRow = kFp8 ? kD : 2 * kD;                // bytes
  static constexpr int kKeyBox = kKeyRow < 128 ? kKeyRow : 128;     // bytes of a key box row
  static constexpr int kKeySlots = kKeyRow <= 128 ? 1 : 2;          // both maps in one, or one each
  static constexpr int kValSlots = kD / 64;                         // 128 value columns each
  static constexpr int kTileSlots = kKeySlots + kValSlots;
  static constexpr int kNS = kNQ < 16 ? 16 : kNQ;                   // columns of S (at least 16)
  static constexpr int kQBytes = kNS * kKeyRow;                     // one map's rows
  // P, N-major: a row of 4 kNQ bf16 per key (map 1 hi, lo, map 2 hi, lo), in blocks of at most
  // 128 bytes.
  static constexpr int kPCols = 4 * kNQ;
  static constexpr int kPRow = kPCols * 2 < 128 ? kPCols * 2 : 128;
  static constexpr int kPBytes = kTile * kPCols * 2;
  static constexpr int kPBufs = kNQ == 32 ? 1 : 2;
  static constexpr int kOCols = kValSlots * kPCols;
  static constexpr int kOBufs = kNQ == 32 && kD == 128 ? 1 : 2;
  static constexpr int kTmemO = 4 * kNS;                            // after two buffers of two S
  static constexpr int kTmemUsed = kTmemO + kOBufs * kOCols;
  static constexpr int kTmemCols = kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
  static_assert(kTmemUsed <= 512, "tensor memory");
};

// Work is laid out on a line: kItemCost steps that hold nothing for each item, then its tiles, a
// step each.  (A segment costs its CTA about as much as two tiles beside its tiles: a CTA with ten
// short items took 91 us where the others took 65.)  `ctas` shares cut the line into `each` or (the
// first `more`) each + 1 steps.  Fewer than 2^31 steps (checked at launch).
struct Shares {
  uint32_t ctas, each, more;
  int32_t mode;  // kPagedWhole, kPagedUncut or kPagedCut
  __device__ __forceinline__ uint32_t begin(uint32_t cta) const {
    return cta * each + min(cta, more);
  }
  __device__ __forceinline__ uint32_t cta_of(uint32_t step) const {
    const uint32_t border = more * (each + 1);
    return step < border ? step / (each + 1) : more + (step - border) / each;
  }
};
// The CTA's share: the item (b, hk, rb) that it begins in, the steps from that item's first one to
// the share's begin and end, and the item's tiles.
struct Share {
  Shares all;
  uint32_t begin;     // of the share
  int32_t off, end;   // from the item's first step; end = off: nothing
  int32_t b, hk, rb, len, units;
};

template <int kNR>
struct Ctrl {
  float m[2][2][kNR];  // reference maxima of both maps' rows, two copies in turn
  float wmax[2][4][kNR];
  float lsum[2][2][4][kNR];  // by segment parity
  float rsum[2][4][kNR];
  float late[2][2][kMaxBad][kNR];  // by segment parity: logits of keys kept out of the product,
  float ref[2][2][kNR];         // and rows' references, by segment parity
  TileDesc ring[kRing], done[2];  // done: a segment's last tile, by segment parity
  RowInfo rows[kRing][kNR];  // by segment
  uint64_t k_full[6], k_empty[6], v_full[6], v_empty[6];
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], pv_done[2], o_empty[2], drain;
  uint32_t bad_rows[3];
  Share share;
  uint32_t tmem;
  int abort, failed;
};

template <int kD, bool kFp8, int kNR>
struct Layout {
  using G = Geo<kD, kFp8, kNR>;
  static constexpr int kP = 0;
  static constexpr int kQ = kP + G::kPBufs * G::kPBytes;
  static constexpr int kFixed = kQ + 4 * G::kQBytes;  // then the ring, then Ctrl
  static constexpr int kRoom =
      227 * 1024 - 1024 - static_cast<int>(sizeof(Ctrl<kNR>)) - kFixed;
  // The ring of keys and that of values: each is filled by a warp of its own and emptied in order.
  static constexpr int kSlots = kRoom / kSlotBytes < 6 ? kRoom / kSlotBytes : 6;
  static constexpr int kShare = kSlots * G::kKeySlots / G::kTileSlots;
  static constexpr int kKeyRing = kShare < G::kKeySlots ? G::kKeySlots : kShare;
  static constexpr int kValRing = kSlots - kKeyRing;
  static_assert(kValRing >= G::kValSlots, "one tile must fit");
  static constexpr int kKeyAt = kFixed, kValAt = kKeyAt + kKeyRing * kSlotBytes;
  static constexpr int kCtrl = kFixed + kSlots * kSlotBytes;
  static constexpr int kBytes = 1024 + kCtrl + static_cast<int>(sizeof(Ctrl<kNR>));
};

__device__ __forceinline__ int32_t units_of(int32_t len, int32_t most) {
  if (len <= 0 || len > most) return 1;  // an idle or invalid sequence still has rows to write
  return (len + kTile - 1) / kTile;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// (A NaN counts only where all are.)
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
// The sums of kN values (a power of two) over the warp; lane l returns that of value
// l / (32 / kN).  Half of the values change hands at each step.
template <int kN>
__device__ __forceinline__ float warp_sums(float (&x)[kN]) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int o = 16, n = kN / 2; o > 0; o >>= 1, n >>= 1) {
    if (n == 0) x[0] += __shfl_xor_sync(0xffffffffu, x[0], o);
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const bool upper = lane & o;
      const float mine = upper ? x[j + n] : x[j], other = upper ? x[j] : x[j + n];
      x[j] = mine + __shfl_xor_sync(0xffffffffu, other, o);
    }
  }
  return x[0];
}

// One arrival on the barrier when this thread's cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void fence_async_proxy() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// tcgen05.mma of a converged warp (one elected lane issues).  The operands' descriptors come as
// their low words (start address, leading-dimension offset), which advance, and their high words
// (stride-dimension offset, layout), which do not: two 32-bit additions a product.
template <bool kFp8>
__device__ __forceinline__ void umma(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t a_hi,
                                     uint32_t b_hi, uint32_t idesc, uint32_t accumulate) {
  if (kFp8)
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %5, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(a_hi), "r"(b_hi), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(a_hi), "r"(b_hi), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ uint32_t low(uint64_t x) { return static_cast<uint32_t>(x); }
__device__ __forceinline__ uint32_t high(uint64_t x) { return static_cast<uint32_t>(x >> 32); }
// Descriptor of rows of 64 bytes with 64-byte swizzle (8-row groups 512 bytes apart): K-major, or
// MN-major operands at most 32 elements wide.
__device__ __forceinline__ uint64_t smem_desc_sw64(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (1ull << 16) |
         (static_cast<uint64_t>(512 >> 4) << 32) | (1ull << 46) | (4ull << 61);
}

// kN consecutive 32-bit tensor-memory columns of the thread's lane; valid after tmem_loaded().
template <int kN>
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[kN]) {
  static_assert(kN == 1 || kN == 2 || kN == 4 || kN == 8, "columns");
  if constexpr (kN == 1)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];"
                 : "=r"(r[0])
                 : "r"(addr)
                 : "memory");
  else if constexpr (kN == 2)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];"
                 : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
  else if constexpr (kN == 4)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
  else
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7]) : "r"(addr) : "memory");
}
// Waits for the thread's loads, passing r through so that no use moves before it.
template <int kN>
__device__ __forceinline__ void tmem_loaded(uint32_t (&r)[kN]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r[0]) : : "memory");
#pragma unroll
  for (int k = 1; k < kN; ++k) asm volatile("" : "+r"(r[k]));
}
template <int kN>
__device__ __forceinline__ void tmem_store(uint32_t addr, const uint32_t (&r)[kN]) {
  if constexpr (kN == 1)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(addr), "r"(r[0])
                 : "memory");
  else if constexpr (kN == 2)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]) : "memory");
  else if constexpr (kN == 4)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
  else
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
        : "memory");
}

// Named barriers beside the softmax warps' 1 and 2.  The key warp finds the share while the other
// warps set up.  The load and query warps wait for that and for the barriers in shared memory, and
// the others, whose bounded waits are for this kernel's own work, until the kernel before has ended.
constexpr uint32_t kLoadBarrier = 3, kStartBarrier = 4;
__device__ __forceinline__ void named_barrier_arrive(uint32_t id, uint32_t count) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// Phase parity of the n-th use (from 0) of buffer n % kBufs.
template <int kBufs>
__device__ __forceinline__ uint32_t phase(uint32_t n) {
  return (n / kBufs) & 1;
}

// The shares of `ctas` CTAs from the sequences' steps: their sum, the most and the least of one
// (per head and row block).
__device__ __forceinline__ Shares cut_line(const FwdParams &p, uint32_t total, uint32_t longest,
                                           uint32_t shortest, uint32_t ctas) {
  const uint32_t heads = p.kv_heads * p.row_blocks, items = p.B * heads, steps = total * heads;
  Shares s;
  s.mode = p.mode;
  s.ctas = min(ctas, steps);
  s.each = steps / s.ctas;
  s.more = steps - s.each * s.ctas;
  if (s.mode != kPagedByLengths) return s;
  if (items <= ctas) {
    const uint64_t tiles = steps - kItemCost * items;
    s.mode = static_cast<uint64_t>(longest - kItemCost) * ctas <= tiles + kMostAlone * ctas
                 ? kPagedWhole
                 : kPagedCut;
  } else {
    // In a share of `most` steps begin at most most / shortest items, rounded up, and what begins
    // last ends at most longest - 1 steps behind it.
    const uint32_t most = s.each + (s.more > 0 ? 1 : 0);
    const uint64_t uncut = min(static_cast<uint64_t>(most - 1 + longest),
                               static_cast<uint64_t>((most - 1) / shortest + 1) * longest);
    s.mode = uncut * ctas <= steps + static_cast<uint64_t>(kUneven) * ctas ? kPagedUncut
                                                                             : kPagedCut;
  }
  return s;
}

// CTA `cta`'s share of `ctas` CTAs (one warp, uniform).
__device__ __forceinline__ Share find_share(const FwdParams &p, uint32_t cta, uint32_t ctas) {
  const int lane = threadIdx.x % 32;
  const int32_t most = p.max_pages * p.page_size;
  Share s = {{1, 1, 0, p.mode}, 0, 0, 0, 0, 0, 0, 0, 1};
  const uint32_t heads = p.kv_heads * p.row_blocks;  // items of a sequence
  int32_t last[4];  // lengths of the last 128 sequences, four a lane
  if (p.mode != kPagedWhole) {
    uint32_t total = 0, longest = 0, shortest = 0xFFFFFFFFu;
#pragma unroll 1
    for (int32_t b0 = 0; b0 < p.B; b0 += 128) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int32_t x = b0 + 32 * k + lane;
        last[k] = x < p.B ? p.kv_len[x] : 0;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (b0 + 32 * k + lane < p.B) {
          const uint32_t u = kItemCost + units_of(last[k], most);
          total += u;
          longest = max(longest, u);
          shortest = min(shortest, u);
        }
    }
    s.all = cut_line(p, __reduce_add_sync(0xffffffffu, total),
                     __reduce_max_sync(0xffffffffu, longest),
                     __reduce_min_sync(0xffffffffu, shortest), ctas);
  }
  if (s.all.mode == kPagedWhole) {
    if (cta < p.B * heads) {
      s.b = cta / heads;
      const uint32_t item = cta - s.b * heads;
      s.hk = item / p.row_blocks;
      s.rb = item - s.hk * p.row_blocks;
      s.len = p.kv_len[s.b];
      s.units = units_of(s.len, most);
      s.end = kItemCost + s.units;
    }
  } else if (cta < s.all.ctas) {
    s.begin = s.all.begin(cta);
    uint32_t left = s.begin;  // steps before the share, counted down sequence by sequence
#pragma unroll 1
    for (int32_t b0 = 0; b0 < p.B; b0 += 32) {
      const int32_t x = b0 + lane;
      const int32_t len = p.B <= 32 ? last[0] : x < p.B ? p.kv_len[x] : 0;
      const uint32_t u = x < p.B ? (kItemCost + units_of(len, most)) * heads : 0;
      uint32_t incl = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const uint32_t all = __shfl_sync(0xffffffffu, incl, 31);
      if (left < all) {
        const int at = __ffs(__ballot_sync(0xffffffffu, left < incl)) - 1;
        s.b = b0 + at;
        left -= __shfl_sync(0xffffffffu, incl - u, at);
        s.len = __shfl_sync(0xffffffffu, len, at);
        break;
      }
      left -= all;
    }
    s.units = units_of(s.len, most);
    const uint32_t item = left / (kItemCost + s.units);
    s.off = static_cast<int32_t>(left - item * (kItemCost + s.units));
    s.end = s.off + static_cast<int32_t>(s.all.each + (cta < s.all.more ? 1 : 0));
    s.hk = item / p.row_blocks;
    s.rb = item - s.hk * p.row_blocks;
  }
  return s;
}

// A load warp's place in its share.  Where items are not cut, a share has those that begin in it.
struct Walk {
  int32_t b, hk, rb, len, units;
  int32_t tile, end;  // the tile, and the share's end, in tiles of the current item
  bool cut;           // items are
  __device__ __forceinline__ Walk(const FwdParams &p, const Share &s)
      : b(s.b), hk(s.hk), rb(s.rb), len(s.len), units(s.units), tile(max(0, s.off - kItemCost)),
        end(s.end - kItemCost), cut(s.all.mode == kPagedCut) {
    if (!cut) {
      if (s.off > 0)
        next_item(p);
      else
        take_whole();
    }
  }
  __device__ __forceinline__ void take_whole() {
    if (!cut && end > -kItemCost) end = max(end, units);
  }
  // To the next item with a tile in the share (the first may be cut before its tiles).
  __device__ __forceinline__ void next_item(const FwdParams &p) {
    end -= units + kItemCost;
    tile = 0;
    if (++rb == p.row_blocks) {
      rb = 0;
      if (++hk == p.kv_heads) {
        hk = 0;
        ++b;
        if (end > (cut ? 0 : -kItemCost)) {
          len = p.kv_len[b];
          units = units_of(len, p.max_pages * p.page_size);
        }
      }
    }
    take_whole();
  }
};

// ---------------------------------------------------------------------------
// The load warps, one for the keys (with the share and the tiles' descriptions) and one for the
// values: a copy takes one thread 80 to 180 cycles to issue, and a tile in pages of 16 rows has 32
// of them, which one warp issues more slowly than HBM delivers.  (Two for the keys alone were no
// faster: 33 us where one takes 30 for 64 x 16 heads of 200 keys.)
// ---------------------------------------------------------------------------
template <int kD, bool kFp8, int kNR, bool kKeys>
__device__ __forceinline__ void load_warp(const FwdParams &p, const CUtensorMap *mk1,
                                          const CUtensorMap *mk2, const CUtensorMap *mv,
                                          uint8_t *smem, Ctrl<kNR> *sm) {
  using G = Geo<kD, kFp8, kNR>;
  using L = Layout<kD, kFp8, kNR>;
  constexpr int kPerTile = kKeys ? G::kKeySlots : G::kValSlots;
  constexpr int kSlots = kKeys ? L::kKeyRing : L::kValRing;
  uint64_t *full = kKeys ? sm->k_full : sm->v_full;
  uint64_t *empty = kKeys ? sm->k_empty : sm->v_empty;
  if (threadIdx.x % 32 == 0) {
    if (kKeys) {
      tma_prefetch_desc(mk1);
      tma_prefetch_desc(mk2);
    } else {
      tma_prefetch_desc(mv);
    }
  }
  // The setup up to here overlaps the kernel before; the kernel after may start its own from here
  // on, so that what it reads before it waits for this one is what this one reads.
  grid_dependency_wait();
  named_barrier_arrive(kStartBarrier, 96 + G::kConsumers);
  // One warp finds the share for the three that walk it, whose copies of the code would have to be
  // fetched too (18 x 8 heads of 100 to 9001 keys 59.9 -> 59.3 us, 152 items of 20 tiles 34.6 ->
  // 33.8).
  if (kKeys) {
    const Share s = find_share(p, blockIdx.x, gridDim.x);
    if (threadIdx.x % 32 == 0) sm->share = s;
    grid_dependents_launch();
  }
  named_barrier_sync(kLoadBarrier, 96 + G::kConsumers);
  Walk w(p, sm->share);
  int32_t &b = w.b, &hk = w.hk, &rb = w.rb, &len = w.len, &units = w.units, &tile = w.tile,
          &end = w.end;
  const int lane = threadIdx.x % 32;
  const int32_t most = p.max_pages * p.page_size;
  // Each slot is two boxes wide and up to eight page pieces high: a lane each.
  const int piece = lane / 2, box = lane % 2;
  const int first_row = piece * p.piece_rows;
  const bool piece_ok = first_row < kTile;
  const auto page_of = [&](int32_t t) {  // this lane's page of tile t of the current sequence
    const int32_t key = t * kTile + first_row;
    return piece_ok && key < len && len <= most
               ? __ldg(p.page_table + static_cast<int64_t>(b) * p.max_pages + p.by_page.div(key))
               : 0;
  };
  bool ok = true;
  uint32_t it = 0;     // tiles
  uint32_t seg = 0;    // segments (the share's parts of items)
  int32_t seg_start = tile;
  int32_t slot = 2 * blockIdx.x;
  int32_t id = tile < end ? page_of(tile) : 0;
  // Read once (by one row block), the pages leave L2 before anything else does.
  const uint64_t policy = p.row_blocks == 1 ? l2_evict_first() : l2_evict_normal();
  uint8_t *ring = smem + (kKeys ? L::kKeyAt : L::kValAt) + box * kBoxBytes;
  const auto freed = [&](uint32_t c) {  // the slot of use c is free again
    return c < kSlots ||
           mbar_wait_warp(&empty[c % kSlots], phase<kSlots>(c - kSlots), &sm->abort, kWaitNs);
  };
#pragma unroll 1
  for (; ok && tile < end; ++it) {
    const bool valid_len = len >= 0 && len <= most;
    const bool seg_last = tile + 1 == units || tile + 1 == end;
    const int32_t page = id, head = hk, key0 = tile * kTile;
    const int32_t tile_len = valid_len ? len : 0;
    const int32_t keys = max(0, min(kTile, tile_len - key0));  // 0 for an idle sequence
    const bool have = piece_ok && first_row < keys;
    const bool bad_id = have && static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.num_pages);
    const int32_t row = p.by_page.mod(key0 + first_row);
    const int32_t z = bad_id ? 0 : page;
    const int32_t rows = (keys + p.piece_rows - 1) & -p.piece_rows;
    const bool seg_first = tile == seg_start;
    TileDesc d;
    int32_t q_row = 0;
    if (kKeys) {
      const bool bad = __any_sync(0xffffffffu, bad_id) || !valid_len;
      d.b = b;
      d.hk = hk;
      d.real = min(kNR, p.rows - rb * kNR);
      d.key0 = key0;
      d.len = tile_len;
      d.slot = slot;
      d.flags = (seg_first ? kFirst : 0) | (seg_last ? kLast : 0) | (bad ? kBad : 0) |
                (seg_start == 0 && tile + 1 == units ? kDirect : 0);
      d.item = (b * p.kv_heads + hk) * p.row_blocks + rb;
      d.steps = max(1, (keys + 15) / 16);
      d.rb = rb;
      q_row = rb * kNR;
      if (bad && lane == 0) report_bad_page(p.status);
    }
    // Move on; the next tile's page numbers are fetched while buffers are awaited.
    if (seg_last) {
      seg_start = 0;
      slot = 2 * blockIdx.x + 1;
    }
    if (++tile == units) w.next_item(p);
    if (tile < end) id = page_of(tile);
#pragma unroll 1
    for (int k = 0; k < kPerTile; ++k) {
      const uint32_t c = it * kPerTile + k;
      const int s = c % kSlots;
      if (!(ok = freed(c))) break;
      // The copies first; their barrier's phase ends no sooner than the arrival below them.
      const int row_bytes = kKeys ? G::kKeyBox : 128;
      if (have) {
        const CUtensorMap *map = !kKeys ? mv : (G::kKeySlots == 1 ? box : k) ? mk2 : mk1;
        const int x = !kKeys ? 128 * k + 64 * box : G::kKeySlots == 1 ? 0 : 64 * box;
        tma_load_4d_hint(ring + s * kSlotBytes + first_row * row_bytes, map, &full[s], x, row, head,
                         z, policy);
      }
      if (kKeys && k == 0) {
        if (lane == 0) sm->ring[it % kRing] = d;
        if (seg_first && lane < kNR) {  // the segment's rows
          const int32_t r = q_row + lane;
          const int32_t i = p.by_group.div(r), pos = tile_len - p.N + i;
          RowInfo info;
          info.last = r >= p.rows || pos < 0 ? -1 : p.causal ? pos : tile_len - 1;
          info.head = d.hk * p.group + r - i * p.group;
          info.out = d.b * p.outs.b + info.head * p.outs.h + i * p.outs.n;
          sm->rows[seg % kRing][lane] = info;
        }
      }
      __syncwarp();
      if (lane == 0) {
        if (rows > 0)
          mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(rows) * 2 * row_bytes);
        else
          mbar_arrive(&full[s]);
      }
    }
    if (kKeys && seg_first) ++seg;
  }
  // The end mark takes the next slot's turn; then the copies still in flight
  // are awaited (bounded), so that none lands after the CTA is gone.
  uint32_t uses = it * kPerTile;
  if (kKeys && ok && freed(uses)) {
    if (lane == 0) {
      sm->ring[it % kRing].flags = kStop;
      mbar_arrive(&full[uses % kSlots]);
    }
    ++uses;
  }
  if (lane == 0) {
    volatile int never = 0;
    for (uint32_t c = uses > kSlots ? uses - kSlots : 0; c < uses; ++c)
      mbar_wait(&full[c % kSlots], phase<kSlots>(c), &never, kDrainNs);
  }
}

// ---------------------------------------------------------------------------
// The query warp: each segment's q rows, 16-byte units into the swizzled operand layout.
// ---------------------------------------------------------------------------
template <int kD, bool kFp8, int kNR>
__device__ __forceinline__ void query_warp(const FwdParams &p, uint8_t *smem, Ctrl<kNR> *sm) {
  using G = Geo<kD, kFp8, kNR>;
  using L = Layout<kD, kFp8, kNR>;
  constexpr int kUnits = G::kKeyRow / 16;
  const int lane = threadIdx.x % 32;
  grid_dependency_wait();
  named_barrier_sync(kLoadBarrier, 96 + G::kConsumers);
  Walk w(p, sm->share);
#pragma unroll 1
  for (uint32_t seg = 0; w.tile < w.end; ++seg) {
    const uint32_t qb = seg & 1;
    if (seg >= 2 && !mbar_wait_warp(&sm->q_empty[qb], phase<2>(seg - 2), &sm->abort, kWaitNs))
      break;
    const int32_t real = min(kNR, p.rows - w.rb * kNR);
#pragma unroll 1
    for (int x = lane; x < 2 * real * kUnits; x += 32) {
      const int map = x >= real * kUnits, y = x - map * real * kUnits;
      const int q = y / kUnits, u = y % kUnits;
      const int r = w.rb * kNR + q;
      const int i = p.by_group.div(r), h = w.hk * p.group + r - i * p.group;
      const diffattn_strides &qs = map ? p.q2s : p.q1s;
      const int64_t at = w.b * qs.b + h * qs.h + i * qs.n;
      const uint8_t *src =
          static_cast<const uint8_t *>(map ? p.q2 : p.q1) + at * (kFp8 ? 1 : 2) + 16 * u;
      uint32_t off;
      if (G::kKeyRow == 64)
        off = q * 64 + ((u ^ ((q >> 1) & 3)) << 4);
      else
        off = (u / 8) * (G::kNS * 128) + q * 128 + (((u % 8) ^ (q & 7)) << 4);
      cp_async16(smem_u32(smem + L::kQ + (2 * qb + map) * G::kQBytes) + off, src);
    }
    cp_async_arrive(&sm->q_full[qb]);
    w.next_item(p);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// ---------------------------------------------------------------------------
// The product warp.
// ---------------------------------------------------------------------------
template <int kD, bool kFp8, int kNR>
__device__ __forceinline__ void mma_warp(const FwdParams &p, uint8_t *smem, Ctrl<kNR> *sm) {
  using G = Geo<kD, kFp8, kNR>;
  using L = Layout<kD, kFp8, kNR>;
  const int lane = threadIdx.x % 32;
  const uint32_t tmem = sm->tmem;
  constexpr uint32_t kIdS = kFp8 ? (1u << 4) | ((G::kNS >> 3) << 17) | ((128u >> 4) << 24)
                                 : idesc_bf16_f32(128, G::kNS, false);
  constexpr uint32_t kIdO = idesc_bf16_f32(128, G::kPCols, true) | (1u << 15);  // both MN-major
  const auto wait = [&](uint64_t *bar, uint32_t parity) {
    return mbar_wait_warp(bar, parity, &sm->abort, kWaitNs);
  };
  const auto ready = [&](uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_test(bar, parity));
  };

  // Tile t's turn in O and tile n's in S; n runs at most one ahead, where its keys are there.
  // The tests see the right phase: the slot's use before was consumed by an earlier tile.
  uint32_t t = 0, n = 0, segs = 0, o_segs = 0;
  int32_t s_flags = 0, o_flags = 0, ahead_flags = 0;  // of S's last tile; of tiles t, t + 1
  int32_t o_steps = 0, ahead_steps = 0;               // 16-key steps with keys in them
  uint64_t since = 0;
#pragma unroll 1
  while (true) {
    const uint32_t cs = n * G::kKeySlots;
    if (n <= t + 1 && !(s_flags & kStop) &&
        ready(&sm->k_full[cs % L::kKeyRing], phase<L::kKeyRing>(cs))) {
      s_flags = *reinterpret_cast<volatile int32_t *>(&sm->ring[n % kRing].flags);
      (n == t ? o_flags : ahead_flags) = s_flags;
      (n == t ? o_steps : ahead_steps) =
          *reinterpret_cast<volatile int32_t *>(&sm->ring[n % kRing].steps);
      if (s_flags & kStop) {
        if (lane == 0) mbar_arrive(&sm->s_full[n & 1]);
      } else {
        if (s_flags & kFirst) {
          if (!wait(&sm->q_full[segs & 1], phase<2>(segs))) break;
          fence_async_proxy();  // the q rows came by ordinary copies
          ++segs;
        }
        tc_fence_after_sync();
        const uint32_t qb = (segs - 1) & 1;
#pragma unroll 1
        for (int map = 0; map < 2; ++map) {
          const uint32_t c = cs + (G::kKeySlots == 2 ? map : 0);
          if (G::kKeySlots == 2 && map == 1 &&
              !wait(&sm->k_full[c % L::kKeyRing], phase<L::kKeyRing>(c)))
            break;
          const uint32_t k_at = smem_u32(smem + L::kKeyAt + (c % L::kKeyRing) * kSlotBytes) +
                                (G::kKeySlots == 1 ? map * kBoxBytes : 0);
          const uint32_t q_at = smem_u32(smem + L::kQ + (2 * qb + map) * G::kQBytes);
          const uint32_t acc = tmem + (n & 1) * 2 * G::kNS + map * G::kNS;
          constexpr bool kNarrow = G::kKeyRow == 64;
          const uint64_t a = kNarrow ? smem_desc_sw64(k_at) : smem_desc_sw128(k_at, 16, 1024);
          const uint64_t b = kNarrow ? smem_desc_sw64(q_at) : smem_desc_sw128(q_at, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < G::kKeyRow / 32; ++kk)  // 32 bytes of depth each
            umma<kFp8>(acc, low(a) + (kk / 4) * (kBoxBytes / 16) + 2 * (kk % 4),
                       low(b) + (kk / 4) * (G::kNS * 8) + 2 * (kk % 4), high(a), high(b), kIdS,
                       kk > 0);
          if (G::kKeySlots == 2 || map == 1) umma_commit_warp(&sm->k_empty[c % L::kKeyRing]);
        }
        if (*reinterpret_cast<volatile int *>(&sm->abort)) break;
        umma_commit_warp(&sm->s_full[n & 1]);
        if (s_flags & kLast) umma_commit_warp(&sm->q_empty[qb]);
      }
      ++n;
      since = 0;
    }
    if (n > t && (o_flags & kStop)) break;
    if (n > t && ready(&sm->p_full[t & 1], phase<2>(t))) {
      if (o_flags & kFirst) {
        // O of the segment before last (this buffer) has been read.
        if (o_segs >= G::kOBufs &&
            !wait(&sm->o_empty[o_segs % G::kOBufs], phase<G::kOBufs>(o_segs - G::kOBufs)))
          break;
        ++o_segs;
      }
      const uint32_t o_at = tmem + G::kTmemO + ((o_segs - 1) % G::kOBufs) * G::kOCols;
      const uint32_t p_at = smem_u32(smem + L::kP + (t % G::kPBufs) * G::kPBytes);
      bool ok = true;
#pragma unroll 1
      for (int k = 0; k < G::kValSlots; ++k) {
        const uint32_t c = t * G::kValSlots + k;
        if (!(ok = wait(&sm->v_full[c % L::kValRing], phase<L::kValRing>(c)))) break;
        tc_fence_after_sync();
        const uint64_t v = smem_desc_sw128(
            smem_u32(smem + L::kValAt + (c % L::kValRing) * kSlotBytes), kBoxBytes, 1024);
        const uint64_t w = G::kPRow == 64 ? smem_desc_sw64(p_at)
                                          : smem_desc_sw128(p_at, kTile * 128, 1024);
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)  // 16 keys each
          if (kk < o_steps)
            umma<false>(o_at + k * G::kPCols, low(v) + 128 * kk, low(w) + G::kPRow * kk, high(v),
                        high(w), kIdO, !(o_flags & kFirst) || kk > 0);
        umma_commit_warp(&sm->v_empty[c % L::kValRing]);
      }
      if (!ok) break;
      umma_commit_warp(&sm->pv_done[t & 1]);
      o_flags = ahead_flags;
      o_steps = ahead_steps;
      ++t;
      since = 0;
      continue;
    }
    // Nothing was ready: bounded, like every wait.
    if (*reinterpret_cast<volatile int *>(&sm->abort)) break;
    if (since == 0) {
      since = globaltimer_ns();
    } else if (globaltimer_ns() - since > kWaitNs) {
      *reinterpret_cast<volatile int *>(&sm->abort) = 1;
      break;
    }
  }
  __syncwarp();
  // Never free tensor memory under a running product.
  umma_commit_warp(&sm->drain);
  volatile int never = 0;
  mbar_wait_warp(&sm->drain, 0, &never, kDrainNs);
}

// ---------------------------------------------------------------------------
// The softmax warps.  Warp w: map (w / 4) % 2, rows by w / 8; its lanes are keys (then value
// columns) 32 (w % 4) + lane of a tile, as tensor memory gives them to it.
// ---------------------------------------------------------------------------
template <int kD, bool kFp8, int kNR>
__device__ __forceinline__ void softmax_warps(const FwdParams &p, uint8_t *smem, Ctrl<kNR> *sm) {
  using G = Geo<kD, kFp8, kNR>;
  using L = Layout<kD, kFp8, kNR>;
  constexpr int kNQ = G::kNQ, kW = G::kW, kChunks = G::kChunks, kMine = G::kMine;
  constexpr int kConsumers = G::kConsumers;
  constexpr int kVUnits = kD / 4;  // 16-byte units of a value row
  const int tid = threadIdx.x - 32 * kSoftmaxWarp, warp = tid / 32, lane = tid % 32;
  const int group = warp / 4, quarter = warp % 4;
  const int map = group & 1, r0 = (group >> 1) * kMine;  // rows r0 .. r0 + kMine - 1
  const int key = 32 * quarter + lane;  // of the tile
  const uint32_t tmem = sm->tmem + (static_cast<uint32_t>(32 * quarter) << 16);
  const auto v_row = [&](uint32_t t, int row, int u) {  // unit u of value row `row` of tile t
    const uint32_t c = t * G::kValSlots + u / 16;
    return reinterpret_cast<uint4 *>(smem + L::kValAt + (c % L::kValRing) * kSlotBytes +
                                     ((u / 8) % 2) * kBoxBytes + row * 128 + (u % 8) * 16);
  };

  float l[kMine];
  int m_turn = 0;
  bool poisoned = false, healthy = true;
  uint32_t late = 0, seg = 0;
  // A segment's end waits for its last product, so it is done after the next tile's P.
  bool pending = false, done_poisoned = false;
  uint32_t done_late = 0;
#pragma unroll 1
  for (uint32_t t = 0;; ++t) {
    bool ok = mbar_wait_warp(&sm->s_full[t & 1], phase<2>(t), &sm->abort, kWaitNs);
    TileDesc d = {};
    if (ok) d = sm->ring[t % kRing];
    const bool stop = !ok || (d.flags & kStop) != 0;
    const int32_t lim_min = p.causal ? d.len - p.N : d.len - 1;  // of a row that sees anything
    const bool masked = d.key0 + kTile - 1 > lim_min;
    const int32_t keys = d.len - d.key0;  // valid rows of the tile if below kTile
    const bool mixed = p.causal && p.N > 1 && masked;  // some rows see keys that others do not
    const int real = kNR == 1 ? 1 : min(d.real - r0, kMine);  // this thread's rows, if above 0
    const RowInfo *rows = sm->rows[seg % kRing] + r0;
    const uint32_t s_at = tmem + (t & 1) * 2 * G::kNS + map * G::kNS + r0;

    const bool fresh = (d.flags & kFirst) != 0;  // nothing in O yet
    const float *m = sm->m[m_turn][map] + r0;

    // This key's products with rows kW k .. (kept in registers while they are few, else read from
    // tensor memory again), and as logits in log2 units, -inf where the key is masked.
    constexpr bool kKeep = kChunks == 1;
    uint32_t raw[kW];
    const auto load = [&](int k) {
      tmem_load(s_at + kW * k, raw);
      tmem_loaded(raw);
    };
    const auto logit = [&](int k, int e) {
      const float x = __uint_as_float(raw[e]) * p.scale_log2;
      return masked && d.key0 + key > rows[kW * k + e].last ? -INFINITY : x;
    };
    // The logits of the loaded rows, for the keys' weights.
    const auto keep_logits = [&](int k) {
      constexpr int kPlane = kNR < 4 ? kNR : 4;
      const int64_t bh = static_cast<int64_t>(d.b) * p.kv_heads + d.hk;
      const int plane = (d.rb * kNR + r0 + kW * k) / kPlane;
      float *dst =
          p.logits + (((bh * 2 + map) * p.planes + plane) * p.padded + d.key0 + key) * kPlane;
#pragma unroll
      for (int e = 0; e < kW; e += kPlane, dst += p.padded * kPlane) {
        if (kW * k + e >= real || !dbg_ok(d.key0 + key < p.padded, p.status, 41)) break;
        if constexpr (kPlane == 1)
          *dst = logit(k, e);
        else if constexpr (kPlane == 2)
          *reinterpret_cast<float2 *>(dst) = make_float2(logit(k, e), logit(k, e + 1));
        else
          *reinterpret_cast<float4 *>(dst) =
              make_float4(logit(k, e), logit(k, e + 1), logit(k, e + 2), logit(k, e + 3));
      }
    };
    bool grew = false;
    if (tid == 0) sm->bad_rows[(t + 1) % 3] = 0;
    if (!stop) {
      if (fresh) {
        poisoned = false;
        late = 0;
#pragma unroll
        for (int q = 0; q < kMine; ++q) l[q] = 0.f;
      }
      if (d.flags & kBad) poisoned = true;
      tc_fence_after_sync();
      float top = -INFINITY;  // how far a logit is above its reference
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        if (kW * k >= real) break;
        load(k);
        if (!fresh) {
          if (masked) {
#pragma unroll
            for (int e = 0; e < kW; ++e) top = fmaxf(top, logit(k, e) - m[kW * k + e]);
          } else {
#pragma unroll
            for (int e = 0; e < kW; ++e)
              top = fmaxf(top, fmaf(__uint_as_float(raw[e]), p.scale_log2, -m[kW * k + e]));
          }
        }
        if (!kKeep && p.logits != nullptr && key < keys) keep_logits(k);
      }
      grew = fresh || top > kGrowth;  // the first tile sets the references
      // P's buffer: the product that read it last is done.
      if (t >= G::kPBufs)
        ok = mbar_wait_warp(&sm->pv_done[(t - G::kPBufs) & 1], phase<2>(t - G::kPBufs), &sm->abort,
                            kWaitNs);
      // Rows of v behind the sequence's end hold anything (NaN too): zero those that the product
      // still takes in its last step of 16, as 0 * NaN would reach every row.  Where new tokens
      // see different keys, a non-finite v row that only some of them see is noted, to be kept out
      // of the product.
      if (ok && (keys < kTile || mixed)) {
        // A wait for a slot's use c is for the right phase only once its use before, c - kValRing,
        // has landed: sure for tiles up to t - kPBufs, whose products are done.  Where a slot may
        // still be tile t - 1's (d = 128, bf16, up to 16 rows), that tile's product is awaited.
        if (L::kValRing < G::kPBufs * G::kValSlots && t > 0)
          ok = mbar_wait_warp(&sm->pv_done[(t - 1) & 1], phase<2>(t - 1), &sm->abort, kWaitNs);
#pragma unroll 1
        for (int k = 0; k < G::kValSlots; ++k) {
          const uint32_t c = t * G::kValSlots + k;
          ok = ok && mbar_wait_warp(&sm->v_full[c % L::kValRing], phase<L::kValRing>(c),
                                    &sm->abort, kWaitNs);
        }
        if (ok) {
          const int from = max(0, keys);
#pragma unroll 1
          for (int k = tid; k < (16 * d.steps - from) * kVUnits; k += kConsumers)
            *v_row(t, from + k / kVUnits, k % kVUnits) = make_uint4(0, 0, 0, 0);
          if (mixed) {
            const int lo = max(0, lim_min + 1 - d.key0), hi = min(kTile, keys);
#pragma unroll 1
            for (int k = tid; k < (hi - lo) * kVUnits; k += kConsumers) {
              const uint4 y = *v_row(t, lo + k / kVUnits, k % kVUnits);
              bool bad = false;
              for (const uint32_t w : {y.x, y.y, y.z, y.w})
                bad |= (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
              const int from_end = d.len - 1 - d.key0 - lo - k / kVUnits;
              if (bad) atomicOr(&sm->bad_rows[t % 3], 1u << from_end);
            }
          }
        }
      }
    }
    ok = ok && healthy;
    if (!ok) *reinterpret_cast<volatile int *>(&sm->failed) = 1;

    // One barrier and vote of all softmax warps: has a logit outgrown its reference (or did a wait
    // run out)?
    if (named_barrier_or(1, kConsumers, grew || !ok)) {
      if (*reinterpret_cast<volatile int *>(&sm->failed)) break;
      if (!stop) {
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
          if (kW * k >= real) break;
          if (!kKeep) load(k);
#pragma unroll
          for (int e = 0; e < kW; ++e) {
            const float y = warp_max(logit(k, e));
            if (lane == 0) sm->wmax[map][quarter][r0 + kW * k + e] = y;
          }
        }
        // O moves with the reference, so the product before must be done.
        if (!fresh)
          ok = mbar_wait_warp(&sm->pv_done[(t - 1) & 1], phase<2>(t - 1), &sm->abort, kWaitNs);
      }
      if (named_barrier_or(2, kConsumers, !ok)) break;
      if (!stop) {
        const auto new_m = [&](int q) {
          float y = fresh ? kLeast : m[q];
#pragma unroll
          for (int w = 0; w < 4; ++w) y = fmaxf(y, sm->wmax[map][w][r0 + q]);
          return y;
        };
        // Rows that are not there never grow.
        if (quarter == 0 && lane < kMine)
          sm->m[m_turn ^ 1][map][r0 + lane] = lane < real ? new_m(lane) : INFINITY;
        if (!fresh) {
          const uint32_t o_at =
              tmem + G::kTmemO + (seg % G::kOBufs) * G::kOCols + map * 2 * kNQ + r0;
          tc_fence_after_sync();
#pragma unroll
          for (int k = 0; k < kChunks; ++k) {
            if (kW * k >= real) break;
            float f[kW];
            bool moved = false;
#pragma unroll
            for (int e = 0; e < kW; ++e) {
              const int q = kW * k + e;
              const float old = m[q], y = new_m(q);
              f[e] = q < real && y != old ? ex2_approx(old - y) : 1.f;
              moved |= q < real && y != old;
              l[q] *= f[e];
            }
            if (moved) {  // the same decision in every thread of the map
#pragma unroll 1
              for (int part = 0; part < 2 * G::kValSlots; ++part) {
                const uint32_t at = o_at + (part / 2) * G::kPCols + (part % 2) * kNQ + kW * k;
                uint32_t y[kW];
                tmem_load(at, y);
                tmem_loaded(y);
#pragma unroll
                for (int e = 0; e < kW; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f[e]);
                tmem_store(at, y);
              }
            }
          }
          tmem_st_wait();
        }
      }
      named_barrier_sync(2, kConsumers);
      m_turn ^= 1;
    }
    if (!stop) {
      // Rows of v to keep out of the product (rare): zero them in the buffer as well, and keep
      // their logits.
      const uint32_t bad_rows = mixed ? sm->bad_rows[t % 3] : 0u;
      const int back = d.len - 1 - d.key0 - key;
      const bool kept_out = bad_rows && back >= 0 && back < kMaxBad && ((bad_rows >> back) & 1);
      if (bad_rows) {
        late |= bad_rows;
#pragma unroll 1
        for (int k = tid; k < kTile * kVUnits; k += kConsumers) {
          const int x_back = d.len - 1 - d.key0 - k / kVUnits;
          if (x_back >= 0 && x_back < kMaxBad && ((bad_rows >> x_back) & 1))
            *v_row(t, k / kVUnits, k % kVUnits) = make_uint4(0, 0, 0, 0);
        }
      }

      // P = 2^(x - m) as bf16 hi + lo.
      uint8_t *p_buf = smem + L::kP + (t % G::kPBufs) * G::kPBytes;
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        if (kW * k >= real) break;
        if (!kKeep) load(k);
        uint32_t hi[kW > 1 ? kW / 2 : 1], lo[kW > 1 ? kW / 2 : 1];
        float y[kW > 1 ? kW : 2];
        y[1] = 0.f;
#pragma unroll
        for (int e = 0; e < kW; ++e) {
          const int q = kW * k + e;
          const float ref = sm->m[m_turn][map][r0 + q];
          if (masked) {
            const float x = logit(k, e);
            if (kept_out) sm->late[seg & 1][map][back][r0 + q] = x;
            y[e] = x == -INFINITY ? 0.f : ex2_approx(x - ref);  // also before any key is seen
          } else {
            y[e] = ex2_approx(fmaf(__uint_as_float(raw[e]), p.scale_log2, -ref));
          }
          l[kW * k + e] += y[e];
        }
#pragma unroll
        for (int e = 0; e < (kW > 1 ? kW / 2 : 1); ++e) {
          hi[e] = pack_bf16x2(y[2 * e], y[2 * e + 1]);
          lo[e] = pack_bf16x2(y[2 * e] - __uint_as_float(hi[e] << 16),
                              y[2 * e + 1] - __uint_as_float(hi[e] & 0xFFFF0000u));
        }
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          const int unit = (map * 2 + part) * (kNQ / 8) + r0 / 8 + k;  // of eight columns
          const uint32_t *src = part ? lo : hi;
          uint8_t *at = p_buf + (unit / 8) * (kTile * 128) + key * G::kPRow +
                        (((unit % 8) ^ (G::kPRow == 64 ? (key >> 1) & 3 : key & 7)) << 4) +
                        2 * (r0 % 8);
          if constexpr (kW == 1)
            *reinterpret_cast<uint16_t *>(at) = static_cast<uint16_t>(src[0]);
          else if constexpr (kW == 2)
            *reinterpret_cast<uint32_t *>(at) = src[0];
          else if constexpr (kW == 4)
            *reinterpret_cast<uint2 *>(at) = make_uint2(src[0], src[1]);
          else
            *reinterpret_cast<uint4 *>(at) = make_uint4(src[0], src[1], src[2], src[3]);
        }
      }
      fence_async_proxy();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->p_full[t & 1]);
      if (kKeep && p.logits != nullptr && key < keys && real > 0) keep_logits(0);
    }

    // ---- the end of the segment before ----
    if (pending) {
      pending = false;
      const RowInfo *done_rows = sm->rows[(seg - 1) % kRing];
      const int parity = (seg - 1) & 1;
      const TileDesc &done = sm->done[parity];
      const int done_real = kNR == 1 ? 1 : done.real;
      const bool direct = (done.flags & kDirect) != 0;
      // A thread has one value column.  The groups of four warps share the rows, kTake at a turn;
      // for d = 128 every other group has the second 128 columns.
      constexpr int kShares = kD == 128 ? G::kSets : 2 * G::kSets;
      constexpr int kTake = kNR / kShares < 1 ? 1 : kNR / kShares < 8 ? kNR / kShares : 8;
      constexpr int kTurns = (kNR + kShares * kTake - 1) / (kShares * kTake);
      constexpr int kHas = kTake * kTurns;
      const int block = kD == 128 ? group & 1 : 0;
      const int share = kD == 128 ? group >> 1 : group;
      const int col = 128 * block + key;
      const auto row_at = [&](int k) { return kTake * (kShares * k + share); };  // of turn k
      const uint32_t o_at =
          tmem + G::kTmemO + ((seg - 1) % G::kOBufs) * G::kOCols + block * G::kPCols;
      // What the output needs from global memory, on its way during the wait.
      constexpr bool kEarly = kHas <= 8;
      float lam[kEarly ? kHas : 1], gain[kEarly ? kHas : 1];
      if (kEarly && direct) {
#pragma unroll
        for (int e = 0; e < kHas; ++e) {
          const int q = row_at(e / kTake) + e % kTake;
          if (q >= done_real) break;
          lam[e] = __ldg(p.lambda + done_rows[q].head);
          gain[e] = p.headnorm && p.norm_w != nullptr
                        ? __ldg(p.norm_w + done_rows[q].head * (2 * kD) + col)
                        : 1.f;
        }
      }
      const uint32_t td = t - 1;
      if (!mbar_wait_warp(&sm->pv_done[td & 1], phase<2>(td), &sm->abort, kWaitNs)) {
        healthy = false;  // the next vote ends the loop
        *reinterpret_cast<volatile int *>(&sm->failed) = 1;
      }
      tc_fence_after_sync();
      const auto l_of = [&](int mp, int q) {
        const float(*x)[kNR] = sm->lsum[parity][mp];
        return (x[0][q] + x[1][q]) + (x[2][q] + x[3][q]);
      };
      float o[kHas];
#pragma unroll
      for (int k = 0; k < kTurns; ++k) {
        const int q0 = row_at(k);
        if (q0 >= done_real) break;
        uint32_t part[4][kTake];  // map 1 hi, lo, map 2 hi, lo
#pragma unroll
        for (int e = 0; e < 4; ++e) tmem_load(o_at + e * kNQ + q0, part[e]);
#pragma unroll
        for (int e = 0; e < 4; ++e) tmem_loaded(part[e]);
        float y[2][kTake];
#pragma unroll
        for (int e = 0; e < kTake; ++e) {
          y[0][e] = __uint_as_float(part[0][e]) + __uint_as_float(part[1][e]);
          y[1][e] = __uint_as_float(part[2][e]) + __uint_as_float(part[3][e]);
        }
        // What the keys kept out of the product add.
#pragma unroll 1
        for (uint32_t rest = done_late; rest; rest &= rest - 1) {
          const int back = __ffs(rest) - 1;
          const int32_t pos = done.len - 1 - back;
          const int32_t page =
              p.page_table[static_cast<int64_t>(done.b) * p.max_pages + p.by_page.div(pos)];
          if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.num_pages)) continue;
          const float v = __bfloat162float(static_cast<const __nv_bfloat16 *>(
              p.v_pages)[page * p.vs.b + done.hk * p.vs.h + p.by_page.mod(pos) * p.vs.n + col]);
#pragma unroll
          for (int e = 0; e < kTake; ++e)
#pragma unroll
            for (int mp = 0; mp < 2; ++mp) {
              const float x = sm->late[parity][mp][back][q0 + e];
              if (x != -INFINITY) y[mp][e] += ex2_approx(x - sm->ref[parity][mp][q0 + e]) * v;
            }
        }
#pragma unroll
        for (int e = 0; e < kTake; ++e) {
          const int q = q0 + e;
          if (q >= done_real) break;
          const float y1 = y[0][e], y2 = y[1][e];
          if (direct) {
            const float lm = kEarly ? lam[kTake * k + e] : __ldg(p.lambda + done_rows[q].head);
            const float z = __fdividef(y1, l_of(0, q)) - lm * __fdividef(y2, l_of(1, q));
            o[kTake * k + e] =
                done_rows[q].last < 0 && !done_poisoned ? 0.f : z;  // 0: the row sees no key
          } else if (dbg_ok(done.slot >= 0 && done.slot < 2 * static_cast<int>(gridDim.x),
                            p.status, 42)) {
            float *dst = p.part + (static_cast<int64_t>(done.slot) * 2 * kNR + q) * (2 * kD) + col;
            dst[0] = y1;
            dst[kNR * (2 * kD)] = y2;
          }
        }
      }
      // The row's (m, l): per slot for the join, per item for the weights.
      if (quarter == 0 && r0 == 0 && (!direct || p.item_ml != nullptr)) {
        float2 *ml = (direct ? p.item_ml + static_cast<int64_t>(done.item) * 2 * kNR
                             : p.part_ml + static_cast<int64_t>(done.slot) * 2 * kNR) +
                     map * kNR;
        if (lane < done_real)
          ml[lane] = make_float2(sm->ref[parity][map][lane],
                                 done_poisoned ? -1.f : l_of(map, lane));
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->o_empty[(seg - 1) % G::kOBufs]);
      if (direct) {
        // Head norm: row sums over the lanes, the four quarters and (d = 128) both halves.
        const auto row_sum = [&](int q) {
          float y =
              (sm->rsum[0][0][q] + sm->rsum[0][1][q]) + (sm->rsum[0][2][q] + sm->rsum[0][3][q]);
          if (kD == 128)
            y += (sm->rsum[1][0][q] + sm->rsum[1][1][q]) + (sm->rsum[1][2][q] + sm->rsum[1][3][q]);
          return y;
        };
#pragma unroll 1
        for (int pass = p.headnorm == 2 ? 0 : 1; pass < 2 && p.headnorm; ++pass) {  // mean, square
#pragma unroll
          for (int k = 0; k < kTurns; ++k) {
            const int q0 = row_at(k);
            if (q0 >= done_real) break;
            float z[kTake];
#pragma unroll
            for (int e = 0; e < kTake; ++e) {
              const float y = q0 + e < done_real ? o[kTake * k + e] : 0.f;
              z[e] = pass ? y * y : y;
            }
            constexpr int kLanes = 32 / kTake;
            const float y = warp_sums(z);
            if (lane % kLanes == 0 && q0 + lane / kLanes < done_real)
              sm->rsum[block][quarter][q0 + lane / kLanes] = y;
          }
          named_barrier_sync(2, kConsumers);
          if (pass == 0) {
#pragma unroll
            for (int k = 0; k < kTurns; ++k) {
              const int q0 = row_at(k);
              if (q0 >= done_real) break;
#pragma unroll
              for (int e = 0; e < kTake; ++e)
                if (q0 + e < done_real) o[kTake * k + e] -= row_sum(q0 + e) * (0.5f / kD);
            }
            named_barrier_sync(2, kConsumers);
          }
        }
#pragma unroll
        for (int k = 0; k < kTurns; ++k) {
          const int q0 = row_at(k);
          if (q0 >= done_real) break;
#pragma unroll
          for (int e = 0; e < kTake; ++e) {
            const int q = q0 + e;
            if (q >= done_real) break;
            float y = o[kTake * k + e];
            if (p.headnorm && (done_rows[q].last >= 0 || done_poisoned)) {
              y *= rsqrtf(row_sum(q) * (0.5f / kD) + p.eps) * p.out_scale;
              if (kEarly)
                y *= gain[kTake * k + e];
              else if (p.norm_w != nullptr)
                y *= __ldg(p.norm_w + done_rows[q].head * (2 * kD) + col);
            }
            p.out[done_rows[q].out + col] = __float2bfloat16_rn(y);
          }
        }
      }
    }
    if (stop) break;
    if (d.flags & kLast) {  // this segment's sums and references, read after the next vote
      constexpr int kLanes = 32 / kMine;
      const float y = warp_sums(l);
      if (lane % kLanes == 0 && lane / kLanes < real)
        sm->lsum[seg & 1][map][quarter][r0 + lane / kLanes] = poisoned ? NAN : y;
      if (quarter == 0 && lane < real)
        sm->ref[seg & 1][map][r0 + lane] = sm->m[m_turn][map][r0 + lane];
      if (tid == 0) sm->done[seg & 1] = d;
      done_poisoned = poisoned;
      done_late = late;
      pending = true;
      ++seg;
    }
  }
}

// The barriers in shared memory (one thread).
template <int kD, bool kFp8, int kNR>
__device__ __forceinline__ void prepare(Ctrl<kNR> *sm) {
  using G = Geo<kD, kFp8, kNR>;
  using L = Layout<kD, kFp8, kNR>;
  for (int s = 0; s < L::kKeyRing; ++s) {
    mbar_init(&sm->k_full[s], 1);
    mbar_init(&sm->k_empty[s], 1);
  }
  for (int s = 0; s < L::kValRing; ++s) {
    mbar_init(&sm->v_full[s], 1);
    mbar_init(&sm->v_empty[s], 1);
  }
  for (int k = 0; k < 2; ++k) {
    mbar_init(&sm->q_full[k], 32);
    mbar_init(&sm->q_empty[k], 1);
    mbar_init(&sm->s_full[k], 1);
    mbar_init(&sm->p_full[k], G::kConsumers / 32);
    mbar_init(&sm->pv_done[k], 1);
    mbar_init(&sm->o_empty[k], G::kConsumers / 32);
  }
  mbar_init(&sm->drain, 1);
  sm->abort = sm->failed = 0;
  for (int k = 0; k < 3; ++k) sm->bad_rows[k] = 0;
  fence_barrier_init();
}

template <int kD, bool kFp8, int kNR>
__global__ void __launch_bounds__(Geo<kD, kFp8, kNR>::kThreads, 1)
    diffpaged_fwd_kernel(const __grid_constant__ CUtensorMap mk1,
                         const __grid_constant__ CUtensorMap mk2,
                         const __grid_constant__ CUtensorMap mv,
                         const __grid_constant__ FwdParams p) {
  using G = Geo<kD, kFp8, kNR>;
  using L = Layout<kD, kFp8, kNR>;
  extern __shared__ uint8_t raw[];
  uint8_t *smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  auto *sm = reinterpret_cast<Ctrl<kNR> *>(smem + L::kCtrl);
  const int warp = threadIdx.x / 32;
  if (warp == kKeyWarp) {
    load_warp<kD, kFp8, kNR, true>(p, &mk1, &mk2, &mv, smem, sm);
  } else if (warp == kValueWarp) {
    load_warp<kD, kFp8, kNR, false>(p, &mk1, &mk2, &mv, smem, sm);
  } else if (warp == kQueryWarp) {
    query_warp<kD, kFp8, kNR>(p, smem, sm);
  } else if (warp == kMmaWarp) {
    tmem_alloc(&sm->tmem, G::kTmemCols);
    tmem_relinquish();
    tc_fence_before_sync();
    named_barrier_sync(kStartBarrier, 96 + G::kConsumers);
    tc_fence_after_sync();
    mma_warp<kD, kFp8, kNR>(p, smem, sm);
  } else if (warp >= kSoftmaxWarp) {
    if (threadIdx.x == 32 * kSoftmaxWarp) prepare<kD, kFp8, kNR>(sm);
    __syncwarp();
    named_barrier_arrive(kLoadBarrier, 96 + G::kConsumers);
    named_barrier_sync(kStartBarrier, 96 + G::kConsumers);
    tc_fence_after_sync();
    softmax_warps<kD, kFp8, kNR>(p, smem, sm);
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(sm->tmem, G::kTmemCols);
  if (threadIdx.x == 0 && *reinterpret_cast<volatile int *>(&sm->abort) && p.status != nullptr)
    atomicExch(p.status, static_cast<int32_t>(DIFFATTN_ERR_TIMEOUT));
}

template <int kD, bool kFp8, int kNR>
diffattn_status launch_main(const FwdParams &p, const CUtensorMap (&maps)[3], int ctas,
                            cudaStream_t stream) {
  constexpr size_t kBytes = Layout<kD, kFp8, kNR>::kBytes;
  static_assert(kBytes <= 227 * 1024, "shared memory of one CTA");
  static std::atomic<bool> attr_set[64];  // per device (concurrent callers may both set)
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DIFFATTN_ERR_CUDA;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(diffpaged_fwd_kernel<kD, kFp8, kNR>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kBytes)) != cudaSuccess)
      return DIFFATTN_ERR_CUDA;
    attr_set[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(Geo<kD, kFp8, kNR>::kThreads);
  cfg.dynamicSmemBytes = kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, diffpaged_fwd_kernel<kD, kFp8, kNR>, maps[0], maps[1], maps[2],
                            p) == cudaSuccess
             ? DIFFATTN_OK
             : DIFFATTN_ERR_CUDA;
}

template <int kD, bool kFp8>
diffattn_status launch_rows(const FwdParams &p, const CUtensorMap (&maps)[3],
                            const PagedFwdPlan &plan, cudaStream_t stream) {
  switch (plan.row_tile) {
    case 1: return launch_main<kD, kFp8, 1>(p, maps, plan.ctas, stream);
    case 2: return launch_main<kD, kFp8, 2>(p, maps, plan.ctas, stream);
    case 4: return launch_main<kD, kFp8, 4>(p, maps, plan.ctas, stream);
    case 8: return launch_main<kD, kFp8, 8>(p, maps, plan.ctas, stream);
    case 16: return launch_main<kD, kFp8, 16>(p, maps, plan.ctas, stream);
    default: return launch_main<kD, kFp8, 32>(p, maps, plan.ctas, stream);
  }
}

}  // namespace

// The main kernel, a file for each head width (paged_fwd_d64.cu, paged_fwd_d128.cu).
diffattn_status launch_paged_main_d64(const FwdParams &p, const CUtensorMap (&maps)[3],
                                      const PagedFwdPlan &plan, bool fp8, cudaStream_t stream);
diffattn_status launch_paged_main_d128(const FwdParams &p, const CUtensorMap (&maps)[3],
                                       const PagedFwdPlan &plan, bool fp8, cudaStream_t stream);

}  // namespace diffattn
