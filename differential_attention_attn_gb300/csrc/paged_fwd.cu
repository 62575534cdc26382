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
// multiply-adds, so up to R = 16 and more this is HBM-bound; everything here
// serves to keep loads in flight.
//
//   - Work is counted in tiles of 64 keys over all sequences and heads, and
//     every CTA (one per SM) takes the same number of consecutive tiles,
//     found from kv_len on the device; a ragged batch is balanced and a graph
//     replays with new lengths.  Items cut by a CTA boundary leave partial
//     states, which a second kernel (launched dependent on the first) joins.
//     With few tiles in all, one CTA takes each item and nothing is joined.
//   - One warp issues TMA copies of page pieces (16, 32 or 64 rows, by the
//     page size) into a ring of tile buffers of about 192 KB.
//   - Eight warps compute: four per map.  S^T = K Q^T by mma.sync (m16n8k16)
//     with the keys as the 16-row operand and 8 rows r as the 8-column one:
//     tcgen05 needs 128 rows per product of which R would be used, while here
//     nothing but the padding to 8 is lost and the tensor pipe stays far from
//     its limit.  The four warps of a map take 16 keys each, exchange P
//     through shared memory and then accumulate a quarter of O^T = V^T P^T.
//   - The reference maximum moves only when some logit passes it by 2^8: one
//     barrier with a vote per tile instead of a reduction.
//   - P enters the second product as bf16 hi + lo (two products, relative
//     error 2^-17): o1 - lambda o2 cancels and the head norm scales the
//     difference back up, so a plain bf16 P would show; the second product is
//     hidden behind the loads.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "debug_check.cuh"
#include "paged.h"
#include "ptx.cuh"

namespace diffattn {
namespace {

constexpr int kTile = kPagedTile;
constexpr int kConsumers = 256;
constexpr int kThreads = kConsumers + 32;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint64_t kDrainNs = 200000000ull;
constexpr float kGrowth = 8.f;  // log2 units a logit may pass the reference maximum by
constexpr int kPStride = kTile + 8;  // bf16 elements of a row of P: 16-byte steps, no bank conflicts
constexpr int kMinShare = 2;  // tiles
constexpr float kLog2e = 1.4426950408889634f;

template <int kD, bool kFp8>
struct Geo {
  static constexpr int kKeyRow = kFp8 ? kD : 2 * kD;               // bytes
  static constexpr int kKeyBox = kKeyRow < 128 ? kKeyRow : 128;    // bytes of a TMA box row
  static constexpr int kKeyBoxes = kKeyRow / kKeyBox;
  static constexpr int kValBoxes = 4 * kD / 128;
  static constexpr int kKeyBytes = kTile * kKeyRow;                // one map's keys of a tile
  static constexpr int kValBytes = kTile * 4 * kD;
  static constexpr int kStageBytes = 2 * kKeyBytes + kValBytes;
  static constexpr int kStages = 196608 / kStageBytes;
  static constexpr int kBoxesPerPiece = 2 * kKeyBoxes + kValBoxes;
};

enum : int32_t { kFirst = 1, kLast = 2, kStop = 4, kBad = 8, kDirect = 16 };

struct TileDesc {
  int32_t b, hk, rb, key0;
  int32_t len, flags, slot, item;
};

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
  int32_t row_blocks, causal, headnorm, whole;
  float eps, out_scale, scale_log2;
  // Workspace (see PagedFwdPlan): partial O [2 C][2][RPB][2 d], their (m, l), one join record per
  // CTA, and for accumulate one record per item, whole items' (m, l) and all logits.
  float *part;
  float2 *part_ml;
  int4 *records;
  int2 *item_records;
  float2 *item_ml;
  float *logits;  // [B * kv_heads][2][rows][padded], log2 units, or null
  int64_t padded;
  float *weights;
};

template <int kD, bool kFp8, int kNT>
struct Smem {
  using G = Geo<kD, kFp8>;
  static constexpr int kRows = 8 * kNT;
  __nv_bfloat16 p[2][2][kRows][kPStride];  // [map][hi, lo]
  float obuf[kRows][2 * kD + 4];
  float wmax[2][4][kRows];
  float lsum[2][4][kRows];
  float rsum[2][4][kRows];
  uint64_t full[G::kStages], empty[G::kStages];
  TileDesc ring[G::kStages];
  unsigned long long bad_rows[3];
  int abort, failed;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// D += A B, A 16 x 16, B 16 x 8, fp32 accumulators.
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two e4m3 values (low half of x, or the high one) as f16x2; exact.
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(x)));
  return r;
}

__device__ __forceinline__ int32_t units_of(int32_t len, int32_t most) {
  if (len <= 0 || len > most) return 1;  // an idle or invalid sequence still has rows to write
  return (len + kTile - 1) / kTile;
}

__device__ __forceinline__ int64_t warp_sum64(int64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ float group_sum(float x) {  // over the 8 lanes with the same lane % 4
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 8);
  x += __shfl_xor_sync(0xffffffffu, x, 16);
  return x;
}

// ---------------------------------------------------------------------------
// The load warp: finds this CTA's tiles, describes them and issues their copies.
// ---------------------------------------------------------------------------
template <int kD, bool kFp8, int kNT>
__device__ void load_warp(const FwdParams &p, const CUtensorMap *mk1, const CUtensorMap *mk2,
                          const CUtensorMap *mv, uint8_t *stages, Smem<kD, kFp8, kNT> *sm) {
  using G = Geo<kD, kFp8>;
  const int lane = threadIdx.x % 32;
  const int32_t most = p.max_pages * p.page_size;
  const int64_t per_unit = static_cast<int64_t>(p.kv_heads) * p.row_blocks;  // items a sequence

  // Where this CTA's share begins: item (b, hk, rb) and tile within it.
  int64_t todo = 0, total = 0, begin = 0, ctas = 1;
  int32_t b = 0, hk = 0, rb = 0, tile = 0, len = 0, units = 1;
  if (p.whole) {
    const uint32_t item = blockIdx.x;
    rb = static_cast<int32_t>(item % p.row_blocks);
    hk = static_cast<int32_t>(item / p.row_blocks % p.kv_heads);
    b = static_cast<int32_t>(item / p.row_blocks / p.kv_heads);
    len = __ldg(p.kv_len + b);
    units = units_of(len, most);
    todo = units;
  } else {
    for (int32_t b0 = 0; b0 < p.B; b0 += 128) {
      int32_t n[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int32_t x = b0 + 32 * k + lane;
        n[k] = x < p.B ? units_of(__ldg(p.kv_len + x), most) : 0;
      }
      total += warp_sum64(static_cast<int64_t>(n[0]) + n[1] + n[2] + n[3]);
    }
    total *= per_unit;
    // Every share has at least kMinShare tiles (the last CTAs may have none).
    ctas = min(static_cast<int64_t>(gridDim.x), max(int64_t{1}, total / kMinShare));
    if (blockIdx.x < ctas) {
      begin = total * blockIdx.x / ctas;
      todo = total * (blockIdx.x + 1) / ctas - begin;
      int64_t left = begin;  // tiles before the share, counted down sequence by sequence
      for (int32_t b0 = 0; b0 < p.B; b0 += 32) {
        const int32_t x = b0 + lane;
        const int64_t u = x < p.B ? units_of(__ldg(p.kv_len + x), most) * per_unit : 0;
        int64_t incl = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        const int64_t all = __shfl_sync(0xffffffffu, incl, 31);
        if (left < all) {
          const int at = __ffs(__ballot_sync(0xffffffffu, left < incl)) - 1;
          b = b0 + at;
          left -= __shfl_sync(0xffffffffu, incl - u, at);
          break;
        }
        left -= all;
      }
      len = __ldg(p.kv_len + b);
      units = units_of(len, most);
      const int32_t item = static_cast<int32_t>(left / units);
      tile = static_cast<int32_t>(left - static_cast<int64_t>(item) * units);
      rb = item % p.row_blocks;
      hk = item / p.row_blocks;
    }
    // The join record of an item that is cut: written by the CTA whose share
    // begins where that of the CTA with the item's first tile ends.
    if (lane == 0) {
      int4 rec = make_int4(-1, 0, 0, 0);
      if (tile > 0) {
        const int64_t start = begin - tile;
        const int64_t c0 = ((start + 1) * ctas - 1) / total;
        if (begin == total * (c0 + 1) / ctas)
          rec = make_int4((b * p.kv_heads + hk) * p.row_blocks + rb,
                          static_cast<int>(2 * c0 + (total * c0 / ctas < start ? 1 : 0)),
                          static_cast<int>(((start + units) * ctas - 1) / total - c0 + 1), 0);
      }
      p.records[blockIdx.x] = rec;
    }
  }

  const int piece = lane / G::kBoxesPerPiece, box = lane % G::kBoxesPerPiece;
  const int pieces = kTile / p.piece_rows;
  const auto page_of = [&](int32_t t) {  // this lane's page of tile t of the current sequence
    const int32_t key = t * kTile + piece * p.piece_rows;
    return piece < pieces && key < len && len <= most
               ? __ldg(p.page_table + static_cast<int64_t>(b) * p.max_pages + key / p.page_size)
               : 0;
  };
  bool ok = true;
  uint32_t it = 0;
  int32_t seg_start = tile;  // first tile of the current segment (the share's part of one item)
  int32_t slot = 2 * blockIdx.x;
  int32_t id = todo > 0 ? page_of(tile) : 0;
  for (int64_t left = todo; left > 0; --left, ++it) {
    const int s = it % G::kStages;
    const bool valid_len = len >= 0 && len <= most;
    const bool seg_last = tile + 1 == units || left == 1;
    const int32_t page = id;
    TileDesc d;
    d.b = b;
    d.hk = hk;
    d.rb = rb;
    d.key0 = tile * kTile;
    d.len = valid_len ? len : 0;
    d.slot = slot;
    d.flags = (tile == seg_start ? kFirst : 0) | (seg_last ? kLast : 0) |
              (seg_start == 0 && tile + 1 == units ? kDirect : 0);
    d.item = (b * p.kv_heads + hk) * p.row_blocks + rb;
    const int32_t keys = max(0, min(kTile, d.len - d.key0));  // 0 for an idle sequence
    const bool have = piece < pieces && piece * p.piece_rows < keys;
    const bool bad_id = have && static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.num_pages);
    const bool bad = __any_sync(0xffffffffu, bad_id) || !valid_len;
    if (bad) d.flags |= kBad;
    if (p.item_records != nullptr && lane == 0 && tile == 0) {
      int32_t n = 1;
      if (!p.whole) {
        const int64_t start = begin + (todo - left);
        n = static_cast<int32_t>(((start + units) * ctas - 1) / total - blockIdx.x + 1);
      }
      p.item_records[d.item] = make_int2(slot, n);
    }
    // Move on; the next tile's page numbers are fetched while a buffer is awaited.
    if (seg_last) {
      seg_start = 0;
      slot = 2 * blockIdx.x + 1;
    }
    if (++tile == units) {
      tile = 0;
      if (++rb == p.row_blocks) {
        rb = 0;
        if (++hk == p.kv_heads) {
          hk = 0;
          ++b;
          if (left > 1) {
            len = __ldg(p.kv_len + b);
            units = units_of(len, most);
          }
        }
      }
    }
    if (left > 1) id = page_of(tile);
    if (it >= G::kStages && !mbar_wait_warp(&sm->empty[s], (it / G::kStages - 1) & 1, &sm->abort,
                                            kWaitNs)) {
      ok = false;
      break;
    }
    uint8_t *buf = stages + s * G::kStageBytes;
    if (lane == 0) {
      if (bad) report_bad_page(p.status);
      sm->ring[s] = d;
      const int32_t rows = (keys + p.piece_rows - 1) / p.piece_rows * p.piece_rows;
      if (rows > 0)
        mbar_arrive_expect_tx(&sm->full[s],
                              static_cast<uint32_t>(rows) * (2 * G::kKeyRow + 4 * kD));
      else
        mbar_arrive(&sm->full[s]);
    }
    __syncwarp();
    if (have) {
      const int32_t row = (d.key0 + piece * p.piece_rows) % p.page_size;
      const int32_t z = bad_id ? 0 : page;
      constexpr int kKeyX = kFp8 ? G::kKeyBox : 64;  // elements of a key box
      const int first_row = piece * p.piece_rows;
      if (box < G::kKeyBoxes) {
        tma_load_4d(buf + (box * kTile + first_row) * G::kKeyBox, mk1, &sm->full[s], box * kKeyX,
                    row, d.hk, z);
      } else if (box < 2 * G::kKeyBoxes) {
        const int x = box - G::kKeyBoxes;
        tma_load_4d(buf + G::kKeyBytes + (x * kTile + first_row) * G::kKeyBox, mk2, &sm->full[s],
                    x * kKeyX, row, d.hk, z);
      } else {
        const int x = box - 2 * G::kKeyBoxes;
        tma_load_4d(buf + 2 * G::kKeyBytes + (x * kTile + first_row) * 128, mv, &sm->full[s],
                    x * 64, row, d.hk, z);
      }
    }
  }
  // The end mark takes the next buffer's turn; then the copies still in flight
  // are awaited (bounded), so that none lands after the CTA is gone.
  if (ok && (it < G::kStages || mbar_wait_warp(&sm->empty[it % G::kStages],
                                               (it / G::kStages - 1) & 1, &sm->abort, kWaitNs))) {
    if (lane == 0) {
      sm->ring[it % G::kStages].flags = kStop;
      mbar_arrive(&sm->full[it % G::kStages]);
    }
    ++it;
  }
  if (lane == 0) {
    volatile int never = 0;
    for (uint32_t k = it > G::kStages ? it - G::kStages : 0; k < it; ++k)
      mbar_wait(&sm->full[k % G::kStages], (k / G::kStages) & 1, &never, kDrainNs);
  }
}

// ---------------------------------------------------------------------------
// The compute warps.  Warp w: map w & 1, quarter w >> 1 (of a tile's keys for
// the first product, of the 2 d value columns for the second).
// Accumulator fragments (16 x 8): lane = 4 g + t holds rows g, g + 8 and
// columns 2 t, 2 t + 1; the rows are keys, then value columns, and the columns
// always the queries 8 nt + 2 t + e of this row block.
// ---------------------------------------------------------------------------
template <int kD, bool kFp8, int kNT>
__device__ void compute_warps(const FwdParams &p, uint8_t *stages, Smem<kD, kFp8, kNT> *sm) {
  using G = Geo<kD, kFp8>;
  constexpr int kRows = 8 * kNT;
  constexpr int kSteps = kD / 16;   // of the first product's depth
  constexpr int kMT = 2 * kD / 64;  // 16-column tiles of a warp's value quarter
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int map = warp & 1, quarter = warp >> 1;
  const int g = lane / 4, t = lane % 4;

  uint32_t q[kSteps][kNT][2];
  float o[kMT][kNT][4];
  float m[kNT][2], l[kNT][2];
  int32_t lim[kNT][2];  // last key that a row sees, -1 for none
  bool poisoned = false;

  for (uint32_t it = 0;; ++it) {
    const int s = it % G::kStages;
    const bool ok = mbar_wait_warp(&sm->full[s], (it / G::kStages) & 1, &sm->abort, kWaitNs);
    TileDesc d = {};
    if (ok) d = sm->ring[s];
    const bool stop = !ok || (d.flags & kStop) != 0;
    uint8_t *buf = stages + s * G::kStageBytes;
    const int32_t lim_min = p.causal ? d.len - p.N : d.len - 1;  // of a row that sees anything
    const bool masked = d.key0 + kTile - 1 > lim_min;
    const int32_t keys = d.len - d.key0;  // valid rows of the tile if below kTile
    const bool mixed = p.causal && p.N > 1 && masked;  // some rows see keys that others do not

    if (!stop && (d.flags & kFirst)) {
      poisoned = false;
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = d.rb * kRows + 8 * nt + 2 * t + e;
          const int i = r / p.group;
          const int32_t pos = d.len - p.N + i;
          lim[nt][e] = r >= p.rows || pos < 0 ? -1 : p.causal ? pos : d.len - 1;
          m[nt][e] = -INFINITY;
          l[nt][e] = 0.f;
        }
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[mt][nt][c] = 0.f;
        // B fragments of q: lane (g, t) holds columns (queries) g, depth 2 t, 2 t + 1, + 8 (e4m3:
        // the four bytes 4 t .. 4 t + 3, the order in which the keys' bytes are taken below).
        const int r = d.rb * kRows + 8 * nt + g;
        const bool real = r < p.rows;
        const int i = real ? r / p.group : 0;
        const int h = d.hk * p.group + (real ? r - i * p.group : 0);
        const diffattn_strides &qs = map ? p.q2s : p.q1s;
        const int64_t at = d.b * qs.b + h * qs.h + i * qs.n;
        const uint8_t *src = static_cast<const uint8_t *>(map ? p.q2 : p.q1) +
                             at * (kFp8 ? 1 : 2);
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks) {
          if (kFp8) {
            const uint32_t x =
                real ? __ldg(reinterpret_cast<const uint32_t *>(src + 16 * ks + 4 * t)) : 0u;
            q[ks][nt][0] = e4m3_pair(x);
            q[ks][nt][1] = e4m3_pair(x >> 16);
          } else {
            q[ks][nt][0] =
                real ? __ldg(reinterpret_cast<const uint32_t *>(src + 32 * ks + 4 * t)) : 0u;
            q[ks][nt][1] =
                real ? __ldg(reinterpret_cast<const uint32_t *>(src + 32 * ks + 4 * t + 16)) : 0u;
          }
        }
      }
    }
    if (d.flags & kBad) poisoned = true;

    // Rows of v behind the sequence's end hold anything (NaN too): zero them, as 0 * NaN would
    // reach every row.  Where new tokens see different keys, a non-finite v row that only some of
    // them see is noted, to be kept out of the product.
    if (threadIdx.x == 0) sm->bad_rows[(it + 1) % 3] = 0;
    if (!stop && keys < kTile) {
      const int from = max(0, keys);
      for (int c = threadIdx.x; c < (kTile - from) * (kD / 4); c += kConsumers) {
        const int row = from + c / (kD / 4), u = c % (kD / 4);
        *reinterpret_cast<uint4 *>(buf + 2 * G::kKeyBytes + ((u / 8) * kTile + row) * 128 +
                                   (u % 8) * 16) = make_uint4(0, 0, 0, 0);
      }
    }
    if (!stop && mixed) {
      const int from = max(0, lim_min + 1 - d.key0), to = min(kTile, keys);
      for (int c = threadIdx.x; c < (to - from) * (kD / 4); c += kConsumers) {
        const int row = from + c / (kD / 4), u = c % (kD / 4);
        const uint4 x = *reinterpret_cast<const uint4 *>(
            buf + 2 * G::kKeyBytes + ((u / 8) * kTile + row) * 128 + (u % 8) * 16);
        bool bad = false;
        for (const uint32_t w : {x.x, x.y, x.z, x.w})
          bad |= (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
        if (bad) atomicOr(&sm->bad_rows[it % 3], 1ull << row);
      }
    }

    // S^T = K Q^T of this warp's 16 keys, in log2 units.
    float x[kNT][4];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int c = 0; c < 4; ++c) x[nt][c] = 0.f;
    bool grew = false;
    if (!stop) {
      const uint32_t keys_at = smem_u32(buf + map * G::kKeyBytes);
      const int row = 16 * quarter + (lane & 15);
      if (!kFp8) {
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks) {
          const int unit = 2 * (ks % 4) + (lane >> 4);
          uint32_t a[4];
          ldsm4(a, keys_at + ((ks / 4) * kTile + row) * 128 + ((unit ^ (row & 7)) << 4));
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) mma_bf16(x[nt], a, q[ks][nt][0], q[ks][nt][1]);
        }
      } else {
#pragma unroll
        for (int kp = 0; kp < kSteps / 2; ++kp) {
          const int unit = 2 * kp + (lane >> 4);
          const int swz = G::kKeyBox == 64 ? (row >> 1) & 3 : row & 7;
          uint32_t w[4];
          ldsm4(w, keys_at + row * G::kKeyBox + ((unit ^ swz) << 4));
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t a[4] = {e4m3_pair(w[2 * k]), e4m3_pair(w[2 * k + 1]),
                                   e4m3_pair(w[2 * k] >> 16), e4m3_pair(w[2 * k + 1] >> 16)};
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
              mma_f16(x[nt], a, q[2 * kp + k][nt][0], q[2 * kp + k][nt][1]);
          }
        }
      }
      const int32_t j = d.key0 + 16 * quarter + g;
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          x[nt][c] *= p.scale_log2;
          if (masked && j + 8 * (c >> 1) > lim[nt][c & 1]) x[nt][c] = -INFINITY;
          grew |= x[nt][c] > m[nt][c & 1] + kGrowth;
        }
      if (p.logits != nullptr) {
        float *dst = p.logits + (static_cast<int64_t>(d.b) * p.kv_heads + d.hk) * 2 * p.rows * p.padded;
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int r = d.rb * kRows + 8 * nt + 2 * t + (c & 1);
            const int32_t key = j + 8 * (c >> 1);
            if (r < p.rows && key < d.len &&
                dbg_ok(key < p.padded, p.status, 41))
              dst[(static_cast<int64_t>(map) * p.rows + r) * p.padded + key] = x[nt][c];
          }
      }
    }
    if (!ok) *reinterpret_cast<volatile int *>(&sm->failed) = 1;

    // One barrier and vote of all eight warps: has a logit outgrown its reference (or did a wait
    // run out)?  It also orders the zeroed rows, and last tile's P, before what follows.
    if (named_barrier_or(1, kConsumers, grew || !ok)) {
      if (*reinterpret_cast<volatile int *>(&sm->failed)) break;
      float w[kNT][2];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float y = fmaxf(x[nt][e], x[nt][e + 2]);
          if (stop) y = -INFINITY;
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
          w[nt][e] = y;
          if (g == 0) sm->wmax[map][quarter][8 * nt + 2 * t + e] = y;
        }
      named_barrier_sync(2, kConsumers);
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float n = m[nt][e];
#pragma unroll
          for (int k = 0; k < 4; ++k) n = fmaxf(n, sm->wmax[map][k][8 * nt + 2 * t + e]);
          const float f = n == m[nt][e] ? 1.f : ex2_approx(m[nt][e] - n);
          m[nt][e] = n;
          l[nt][e] *= f;
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt) {
            o[mt][nt][e] *= f;
            o[mt][nt][e + 2] *= f;
          }
        }
    }
    if (stop) break;

    // Rows of v to keep out of the product (rare): zero them in the buffer as well.
    const unsigned long long bad_rows = mixed ? sm->bad_rows[it % 3] : 0ull;
    if (bad_rows) {
      for (int c = threadIdx.x; c < kTile * (kD / 4); c += kConsumers) {
        const int row = c / (kD / 4), u = c % (kD / 4);
        if ((bad_rows >> row) & 1)
          *reinterpret_cast<uint4 *>(buf + 2 * G::kKeyBytes + ((u / 8) * kTile + row) * 128 +
                                     (u % 8) * 16) = make_uint4(0, 0, 0, 0);
      }
      named_barrier_sync(2, kConsumers);
    }

    // P = 2^(x - m), into shared memory as bf16 hi + lo, [query][key].
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int e = c & 1, key = 16 * quarter + g + 8 * (c >> 1);
        float y = ex2_approx(x[nt][c] - m[nt][e]);
        if (masked && d.key0 + key > lim[nt][e]) y = 0.f;
        l[nt][e] += y;
        const __nv_bfloat16 hi = __float2bfloat16_rn(y);
        sm->p[map][0][8 * nt + 2 * t + e][key] = hi;
        sm->p[map][1][8 * nt + 2 * t + e][key] = __float2bfloat16_rn(y - __bfloat162float(hi));
      }
    named_barrier_sync(3 + map, kConsumers / 2);

    // O^T += V^T P^T over the tile's 64 keys, this warp's quarter of the columns.
    const uint32_t v_at = smem_u32(buf + 2 * G::kKeyBytes);
#pragma unroll
    for (int half = 0; half < 2; ++half) {  // 32 keys
      uint32_t ph[kNT][4], pl[kNT][4];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        const int row = 8 * nt + (lane & 7), unit = 4 * half + (lane >> 3);
        ldsm4(ph[nt], smem_u32(&sm->p[map][0][row][8 * unit]));
        ldsm4(pl[nt], smem_u32(&sm->p[map][1][row][8 * unit]));
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {  // 16 keys
        const int row = 32 * half + 16 * k + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
          const int unit = (quarter * kMT + mt) * 2 + ((lane >> 3) & 1);  // of 8 columns
          uint32_t a[4];
          ldsm4_t(a, v_at + ((unit / 8) * kTile + row) * 128 + (((unit % 8) ^ (row & 7)) << 4));
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) {
            mma_bf16(o[mt][nt], a, ph[nt][2 * k], ph[nt][2 * k + 1]);
            mma_bf16(o[mt][nt], a, pl[nt][2 * k], pl[nt][2 * k + 1]);
          }
        }
      }
    }
    if (bad_rows) {  // the kept-out rows, for the queries that do see them
      for (int row = 0; row < kTile; ++row) {
        if (!((bad_rows >> row) & 1)) continue;
        const int32_t key = d.key0 + row;
        const int32_t page =
            p.page_table[static_cast<int64_t>(d.b) * p.max_pages + key / p.page_size];
        if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.num_pages)) continue;
        const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(p.v_pages) +
                                 page * p.vs.b + d.hk * p.vs.h +
                                 (key % p.page_size) * p.vs.n;
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (key > lim[nt][e]) continue;
            const int r = 8 * nt + 2 * t + e;
            const float y = __bfloat162float(sm->p[map][0][r][row]) +
                            __bfloat162float(sm->p[map][1][r][row]);
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt) {
              const int col = (quarter * kMT + mt) * 16 + g;
              o[mt][nt][e] += y * __bfloat162float(v[col]);
              o[mt][nt][e + 2] += y * __bfloat162float(v[col + 8]);
            }
          }
      }
    }
    if (keys < kTile || bad_rows)  // ordinary stores before the next copy into this buffer
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm->empty[s]);
    if (!(d.flags & kLast)) continue;

    // ---- end of the segment ----
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float y = group_sum(l[nt][e]);
        if (g == 0) sm->lsum[map][quarter][8 * nt + 2 * t + e] = y;
      }
    named_barrier_sync(2, kConsumers);
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float y = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) y += sm->lsum[map][k][8 * nt + 2 * t + e];
        l[nt][e] = poisoned ? NAN : y;
      }
    const bool direct = (d.flags & kDirect) != 0;
    // The row's (m, l): per slot for the join, per item for the weights.
    if (quarter == 0 && g == 0 && (!direct || p.item_ml != nullptr)) {
      float2 *ml = direct ? p.item_ml + static_cast<int64_t>(d.item) * 2 * kRows
                          : p.part_ml + static_cast<int64_t>(d.slot) * 2 * kRows;
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          ml[map * kRows + 8 * nt + 2 * t + e] = make_float2(m[nt][e], l[nt][e]);
    }
    if (!direct) {
      float *dst = p.part + (static_cast<int64_t>(d.slot) * 2 + map) * kRows * (2 * kD);
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int r = 8 * nt + 2 * t + (c & 1);
          if (d.rb * kRows + r >= p.rows) continue;
          if (!dbg_ok(d.slot >= 0 && d.slot < 2 * static_cast<int>(gridDim.x), p.status, 42))
            continue;
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt)
            dst[r * (2 * kD) + (quarter * kMT + mt) * 16 + g + 8 * (c >> 1)] = o[mt][nt][c];
        }
      continue;
    }
    // Whole item: map 2's warps hand over -lambda o2, map 1's form o, its norm and the output.
    if (map == 1) {
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = d.rb * kRows + 8 * nt + 2 * t + e;
          if (r >= p.rows) continue;
          const float f = -__ldg(p.lambda + d.hk * p.group + r % p.group) / l[nt][e];
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt) {
            const int col = (quarter * kMT + mt) * 16 + g;
            sm->obuf[8 * nt + 2 * t + e][col] = f * o[mt][nt][e];
            sm->obuf[8 * nt + 2 * t + e][col + 8] = f * o[mt][nt][e + 2];
          }
        }
    }
    named_barrier_sync(2, kConsumers);
    if (map == 1) continue;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool real = d.rb * kRows + 8 * nt + 2 * t + e < p.rows;
        const float f = 1.f / l[nt][e];
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
          const int col = (quarter * kMT + mt) * 16 + g;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float &y = o[mt][nt][e + 2 * k];
            y = real ? fmaf(f, y, sm->obuf[8 * nt + 2 * t + e][col + 8 * k]) : 0.f;
            if (lim[nt][e] < 0 && !poisoned) y = 0.f;  // a row that sees no key
          }
        }
      }
    // Row sums over the 2 d columns: this lane's, its warp's, the four warps'.
    const auto row_sums = [&](float (&tot)[kNT][2]) {
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          tot[nt][e] = group_sum(tot[nt][e]);
          if (g == 0) sm->rsum[0][quarter][8 * nt + 2 * t + e] = tot[nt][e];
        }
      named_barrier_sync(3, kConsumers / 2);
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          tot[nt][e] = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) tot[nt][e] += sm->rsum[0][k][8 * nt + 2 * t + e];
        }
      named_barrier_sync(3, kConsumers / 2);
    };
    float gain[kNT][2];
    if (p.headnorm == 2) {
      float mean[kNT][2];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mean[nt][e] = 0.f;
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt) mean[nt][e] += o[mt][nt][e] + o[mt][nt][e + 2];
        }
      row_sums(mean);
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt) o[mt][nt][c] -= mean[nt][c & 1] * (0.5f / kD);
    }
    if (p.headnorm) {
      float sq[kNT][2];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sq[nt][e] = 0.f;
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt)
            sq[nt][e] += o[mt][nt][e] * o[mt][nt][e] + o[mt][nt][e + 2] * o[mt][nt][e + 2];
        }
      row_sums(sq);
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          gain[nt][e] = rsqrtf(sq[nt][e] * (0.5f / kD) + p.eps) * p.out_scale;
    }
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = d.rb * kRows + 8 * nt + 2 * t + e;
        if (r >= p.rows) continue;
        const int i = r / p.group, h = d.hk * p.group + r - i * p.group;
        __nv_bfloat16 *dst = p.out + d.b * p.outs.b + h * p.outs.h + i * p.outs.n;
        const bool none = lim[nt][e] < 0 && !poisoned;
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int col = (quarter * kMT + mt) * 16 + g + 8 * k;
            float y = o[mt][nt][e + 2 * k];
            if (p.headnorm && !none) {
              y *= gain[nt][e];
              if (p.norm_w != nullptr) y *= __ldg(p.norm_w + h * (2 * kD) + col);
            }
            dst[col] = __float2bfloat16_rn(y);
          }
      }
  }
}

template <int kD, bool kFp8, int kNT>
__global__ void __launch_bounds__(kThreads, 1)
    diffpaged_fwd_kernel(const __grid_constant__ CUtensorMap mk1,
                         const __grid_constant__ CUtensorMap mk2,
                         const __grid_constant__ CUtensorMap mv,
                         const __grid_constant__ FwdParams p) {
  using G = Geo<kD, kFp8>;
  extern __shared__ uint8_t raw[];
  uint8_t *stages = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  auto *sm = reinterpret_cast<Smem<kD, kFp8, kNT> *>(stages + G::kStages * G::kStageBytes);
  grid_dependents_launch();
  if (threadIdx.x == kConsumers) {
    for (int s = 0; s < G::kStages; ++s) {
      mbar_init(&sm->full[s], 1);
      mbar_init(&sm->empty[s], kConsumers / 32);
    }
    sm->abort = sm->failed = 0;
    for (int k = 0; k < 3; ++k) sm->bad_rows[k] = 0;
    fence_barrier_init();
  }
  __syncthreads();
  if (threadIdx.x >= kConsumers)
    load_warp<kD, kFp8, kNT>(p, &mk1, &mk2, &mv, stages, sm);
  else
    compute_warps<kD, kFp8, kNT>(p, stages, sm);
  __syncthreads();
  if (threadIdx.x == 0 && *reinterpret_cast<volatile int *>(&sm->abort) && p.status != nullptr)
    atomicExch(p.status, static_cast<int32_t>(DIFFATTN_ERR_TIMEOUT));
}

// ---------------------------------------------------------------------------
// The second kernel: joins the items that a CTA boundary cut and adds the
// keys' weights.  Launched dependent on the first, whose end it awaits.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;
constexpr int kWeightKeys = 4 * kJoinThreads;  // keys per weight block, four a thread

struct JoinParams {
  FwdParams f;
  int32_t ctas, join_rows, row_tile;  // row_tile: rows of a block of the main kernel
  int32_t weight_chunks;              // per (sequence, key/value head); 0 without weights
};

__device__ __forceinline__ float block_sum(float x, float *scratch) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if (threadIdx.x % 32 == 0) scratch[threadIdx.x / 32] = x;
  __syncthreads();
  float y = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) y += scratch[w];
  __syncthreads();
  return y;
}

// Slot of the k-th part of an item whose first part has slot `first`.
__device__ __forceinline__ int part_slot(int first, int k) {
  return k == 0 ? first : 2 * (first / 2 + k);
}

__device__ __forceinline__ bool parts_ok(int first, int n, int ctas) {
  return first >= 0 && n >= 1 && first / 2 + n <= ctas;
}

// Block (boundary, row): one row of the item cut at that boundary.
template <int kD>
__device__ void join_row(const JoinParams &jp, bool timed_out) {
  const FwdParams &p = jp.f;
  __shared__ float factor[2][512];
  __shared__ float scratch[kJoinThreads / 32];
  __shared__ float half[2][2 * kD];
  const int boundary = 1 + blockIdx.x / jp.join_rows, row = blockIdx.x % jp.join_rows;
  const int4 rec = p.records[boundary];
  if (rec.x < 0 || !parts_ok(rec.y, rec.z, jp.ctas) || rec.z > 512) return;
  const int rb = rec.x % p.row_blocks, bh = rec.x / p.row_blocks;
  const int hk = bh % p.kv_heads, b = bh / p.kv_heads;
  const int r = rb * jp.row_tile + row;
  if (r >= p.rows) return;
  const int i = r / p.group, h = hk * p.group + r - i * p.group;
  const int n = rec.z;

  // Factors 2^(m_s - M) / l, l = sum 2^(m_s - M) l_s, of both maps: warps 0 and 1.
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (warp < 2) {
    float top = -INFINITY, sum = 0.f;
    for (int k = lane; k < n; k += 32)
      top = fmaxf(top, p.part_ml[(part_slot(rec.y, k) * 2ll + warp) * jp.row_tile + row].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    for (int k = lane; k < n; k += 32) {
      const float2 ml = p.part_ml[(part_slot(rec.y, k) * 2ll + warp) * jp.row_tile + row];
      const float f = ml.x == top ? 1.f : exp2f(ml.x - top);
      factor[warp][k] = f;
      sum += f * ml.y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float c = (warp ? -__ldg(p.lambda + h) : 1.f) / sum;
    for (int k = lane; k < n; k += 32) factor[warp][k] *= c;
  }
  __syncthreads();
  constexpr int kGroups = kJoinThreads / (2 * kD);  // threads per column: 2 (d = 64) or 1
  const int col = threadIdx.x % (2 * kD), part = threadIdx.x / (2 * kD);
  const float *src = p.part + static_cast<int64_t>(row) * (2 * kD) + col;
  const int64_t map_step = static_cast<int64_t>(jp.row_tile) * (2 * kD);
  float o = 0.f;
#pragma unroll 4
  for (int k = part; k < n; k += kGroups) {
    const float *x = src + part_slot(rec.y, k) * 2 * map_step;
    o = fmaf(factor[0][k], x[0], fmaf(factor[1][k], x[map_step], o));
  }
  if (kGroups == 2) {
    half[part][col] = o;
    __syncthreads();
    o = half[0][col] + half[kGroups - 1][col];
  }
  const int32_t len = p.kv_len[b];
  if (len - p.N + i < 0) o = 0.f;  // padding: sees no key (the factors are not numbers)
  const float mine = part == 0 ? 1.f : 0.f;  // each column counted once
  if (p.headnorm == 2) o -= block_sum(mine * o, scratch) * (0.5f / kD);
  if (p.headnorm) {
    const float ss = block_sum(mine * o * o, scratch);
    float y = rsqrtf(ss * (0.5f / kD) + p.eps) * p.out_scale;
    if (p.norm_w != nullptr) y *= __ldg(p.norm_w + h * (2 * kD) + col);
    o = len - p.N + i < 0 ? 0.f : o * y;
  }
  if (part == 0)
    p.out[b * p.outs.b + h * p.outs.h + i * p.outs.n + col] =
        __float2bfloat16_rn(timed_out ? NAN : o);
}

// Block (sequence, key/value head, 1024 keys): weights[j] += sum_r |map1 - lambda map2|.
__device__ void add_weights(const JoinParams &jp, int64_t block) {
  const FwdParams &p = jp.f;
  extern __shared__ float4 row_stat[];  // per row: M1, 1 / l1, M2, lambda / l2
  const int chunk = static_cast<int>(block % jp.weight_chunks);
  const int bh = static_cast<int>(block / jp.weight_chunks);
  const int hk = bh % p.kv_heads, b = bh / p.kv_heads;
  const int32_t len = __ldg(p.kv_len + b);
  if (len < 0 || len > p.max_pages * p.page_size || chunk * kWeightKeys >= len) return;
  const int32_t *table = p.page_table + static_cast<int64_t>(b) * p.max_pages;
  bool bad = false;
  for (int k = threadIdx.x; k * p.page_size < len; k += kJoinThreads)
    bad |= static_cast<uint32_t>(__ldg(table + k)) >= static_cast<uint32_t>(p.num_pages);
  if (__syncthreads_or(bad)) return;  // the sequence's weights stay as they are
  for (int k = threadIdx.x; k < 2 * p.rows; k += kJoinThreads) {
    const int map = k & 1, r = k >> 1;
    const int item = bh * p.row_blocks + r / jp.row_tile, row = r % jp.row_tile;
    const int2 rec = p.item_records[item];
    float top, sum;
    if (rec.y == 1) {
      const float2 ml = p.item_ml[(item * 2ll + map) * jp.row_tile + row];
      top = ml.x;
      sum = ml.y;
    } else {
      top = -INFINITY;
      sum = 0.f;
      const int n = parts_ok(rec.x, rec.y, jp.ctas) ? rec.y : 0;
      for (int s = 0; s < n; ++s)
        top = fmaxf(top, p.part_ml[(part_slot(rec.x, s) * 2ll + map) * jp.row_tile + row].x);
      for (int s = 0; s < n; ++s) {
        const float2 ml = p.part_ml[(part_slot(rec.x, s) * 2ll + map) * jp.row_tile + row];
        sum = fmaf(ml.x == top ? 1.f : exp2f(ml.x - top), ml.y, sum);
      }
    }
    const bool none = len - p.N + r / p.group < 0;  // the row sees no key: it adds nothing
    float *dst = reinterpret_cast<float *>(row_stat + r) + 2 * map;
    dst[0] = none ? 0.f : top;
    dst[1] = none ? 0.f : (map ? __ldg(p.lambda + hk * p.group + r % p.group) : 1.f) / sum;
  }
  __syncthreads();
  const int32_t key = chunk * kWeightKeys + 4 * static_cast<int32_t>(threadIdx.x);
  if (key >= len) return;
  const float *x1 = p.logits + static_cast<int64_t>(bh) * 2 * p.rows * p.padded + key;
  const float *x2 = x1 + p.rows * p.padded;
  float w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int r = 0; r < p.rows; ++r) {
    const float4 a = *reinterpret_cast<const float4 *>(x1 + r * p.padded);
    const float4 c = *reinterpret_cast<const float4 *>(x2 + r * p.padded);
    const float4 st = row_stat[r];
    if (st.y == 0.f) continue;
    w[0] += fabsf(exp2f(a.x - st.x) * st.y - exp2f(c.x - st.z) * st.w);
    w[1] += fabsf(exp2f(a.y - st.x) * st.y - exp2f(c.y - st.z) * st.w);
    w[2] += fabsf(exp2f(a.z - st.x) * st.y - exp2f(c.z - st.z) * st.w);
    w[3] += fabsf(exp2f(a.w - st.x) * st.y - exp2f(c.w - st.z) * st.w);
  }
  const int32_t page = __ldg(table + key / p.page_size);
  float *dst = p.weights + (static_cast<int64_t>(page) * p.kv_heads + hk) * p.page_size +
               key % p.page_size;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (key + k < len) dst[k] += w[k];
}

template <int kD>
__global__ void __launch_bounds__(kJoinThreads)
    diffpaged_join_kernel(const __grid_constant__ JoinParams jp) {
  grid_dependency_wait();
  const bool timed_out =
      jp.f.status != nullptr &&
      *reinterpret_cast<volatile const int32_t *>(jp.f.status) == DIFFATTN_ERR_TIMEOUT;
  const int64_t joins = static_cast<int64_t>(jp.ctas - 1) * jp.join_rows;
  if (blockIdx.x < joins)
    join_row<kD>(jp, timed_out);
  else if (!timed_out)
    add_weights(jp, blockIdx.x - joins);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// A pool {width, page_size, heads, pages}: boxes of `rows` rows and at most 128 bytes.
bool encode_pool(CUtensorMap *map, const void *base, int64_t width, const diffpaged_cache &c,
                 const diffattn_strides &st, bool fp8, int rows) {
  static EncodeTiledFn encode = [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<EncodeTiledFn>(ptr);
  }();
  if (encode == nullptr) return false;
  const cuuint64_t es = fp8 ? 1 : 2;
  const cuuint32_t box_x = fp8 && width > 128 ? 128 : fp8 ? static_cast<cuuint32_t>(width) : 64;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(c.page_size),
                              static_cast<cuuint64_t>(c.kv_heads),
                              static_cast<cuuint64_t>(c.num_pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(st.n) * es,
                                 static_cast<cuuint64_t>(st.h) * es,
                                 static_cast<cuuint64_t>(st.b) * es};
  const cuuint32_t box[4] = {box_x, static_cast<cuuint32_t>(rows), 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return encode(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                const_cast<void *>(base), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE,
                box_x * es == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kD, bool kFp8, int kNT>
diffattn_status launch_main(const FwdParams &p, const CUtensorMap (&maps)[3], int ctas,
                            cudaStream_t stream) {
  using G = Geo<kD, kFp8>;
  constexpr size_t kBytes = 1024 + G::kStages * G::kStageBytes + sizeof(Smem<kD, kFp8, kNT>);
  static_assert(kBytes <= 227 * 1024, "shared memory of one CTA");
  static std::atomic<bool> attr_set[64];  // per device (concurrent callers may both set)
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DIFFATTN_ERR_CUDA;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(diffpaged_fwd_kernel<kD, kFp8, kNT>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kBytes)) != cudaSuccess)
      return DIFFATTN_ERR_CUDA;
    attr_set[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kBytes;
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, diffpaged_fwd_kernel<kD, kFp8, kNT>, maps[0], maps[1], maps[2],
                            p) == cudaSuccess
             ? DIFFATTN_OK
             : DIFFATTN_ERR_CUDA;
}

template <int kD>
diffattn_status launch_join(const JoinParams &jp, cudaStream_t stream) {
  const int64_t blocks = static_cast<int64_t>(jp.ctas - 1) * jp.join_rows +
                         static_cast<int64_t>(jp.f.B) * jp.f.kv_heads * jp.weight_chunks;
  if (blocks == 0) return DIFFATTN_OK;
  if (blocks > INT32_MAX) return DIFFATTN_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = jp.weight_chunks ? sizeof(float4) * jp.f.rows : 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, diffpaged_join_kernel<kD>, jp) == cudaSuccess ? DIFFATTN_OK
                                                                               : DIFFATTN_ERR_CUDA;
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

bool plan_paged_fwd(const diffattn_desc &desc, const diffpaged_cache &cache, bool accumulate,
                    int sm_count, PagedFwdPlan *plan) {
  PagedFwdPlan &q = *plan;
  q = PagedFwdPlan{};
  const int64_t rows = desc.N * (desc.H / cache.kv_heads);
  q.row_tiles = rows <= 8 ? 1 : 2;
  const int64_t row_tile = 8 * q.row_tiles;
  q.row_blocks = static_cast<int>((rows + row_tile - 1) / row_tile);
  const double items = static_cast<double>(desc.B) * static_cast<double>(cache.kv_heads) * q.row_blocks;
  if (items > INT32_MAX) return false;
  q.items = desc.B * cache.kv_heads * q.row_blocks;
  const int64_t most = cache.max_pages * cache.page_size;
  const int64_t units = (most + kTile - 1) / kTile;
  q.padded = units * kTile;
  // One CTA per item where no item can have more tiles than the join's launch would cost.
  q.whole = units <= 4;
  q.ctas = q.whole ? static_cast<int>(q.items) : sm_count;
  if (!q.whole && q.items * units < sm_count) q.ctas = static_cast<int>(q.items * units);
  const size_t slots = q.whole ? 0 : 2 * static_cast<size_t>(q.ctas);
  size_t at = 0;
  const auto take = [&at](size_t bytes) {
    const size_t here = at;
    at += round256(bytes);
    return here;
  };
  q.part = take(slots * 2 * row_tile * 2 * desc.d * sizeof(float));
  q.stats = take(slots * 2 * row_tile * sizeof(float2));
  q.records = take(q.whole ? 0 : q.ctas * sizeof(int4));
  if (accumulate) {
    const double logits = static_cast<double>(desc.B) * static_cast<double>(cache.kv_heads) * 2.0 *
                          static_cast<double>(rows) * static_cast<double>(q.padded) * 4.0;
    if (logits > 1.0e18) return false;
    q.items_rec = take(q.items * sizeof(int2));
    q.item_stats = take(q.items * 2 * row_tile * sizeof(float2));
    q.logits = take(static_cast<size_t>(desc.B * cache.kv_heads * 2 * rows * q.padded) * sizeof(float));
  }
  q.bytes = at;
  return true;
}

diffattn_status launch_paged_fwd(const diffattn_desc &desc, const diffpaged_cache &cache,
                                 const PagedFwdPlan &plan, const void *q1, const void *q2,
                                 const float *lambda, const float *norm_w, void *out,
                                 const diffattn_strides *strides, bool accumulate,
                                 void *workspace, cudaStream_t stream) {
  const bool fp8 = desc.dtype == DIFFATTN_E4M3_QK;
  const int64_t d = desc.d, N = desc.N, H = desc.H;
  FwdParams p = {};
  p.q1 = q1;
  p.q2 = q2;
  p.v_pages = cache.v;
  p.lambda = lambda;
  p.norm_w = norm_w;
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.page_table = cache.page_table;
  p.kv_len = cache.kv_len;
  p.status = desc.status_dev;
  p.q1s = strides ? strides[0] : diffattn_strides{H * N * d, N * d, d};
  p.q2s = strides ? strides[1] : p.q1s;
  p.outs = strides ? strides[2] : diffattn_strides{H * N * 2 * d, N * 2 * d, 2 * d};
  p.vs = cache.v_strides;
  p.B = static_cast<int32_t>(desc.B);
  p.H = static_cast<int32_t>(H);
  p.N = static_cast<int32_t>(N);
  p.kv_heads = static_cast<int32_t>(cache.kv_heads);
  p.group = p.H / p.kv_heads;
  p.rows = p.N * p.group;
  p.num_pages = static_cast<int32_t>(cache.num_pages);
  p.max_pages = static_cast<int32_t>(cache.max_pages);
  p.page_size = cache.page_size;
  p.piece_rows = cache.page_size % 64 == 0 ? 64 : cache.page_size % 32 == 0 ? 32 : 16;
  p.row_blocks = plan.row_blocks;
  p.causal = desc.causal ? 1 : 0;
  p.headnorm = desc.headnorm;
  p.whole = plan.whole ? 1 : 0;
  p.eps = desc.eps;
  p.out_scale = 1.0f - desc.lambda_init;
  p.scale_log2 = kLog2e / std::sqrt(static_cast<float>(d));
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  if (!plan.whole) {
    p.part = reinterpret_cast<float *>(ws + plan.part);
    p.part_ml = reinterpret_cast<float2 *>(ws + plan.stats);
    p.records = reinterpret_cast<int4 *>(ws + plan.records);
  }
  if (accumulate) {
    p.item_records = reinterpret_cast<int2 *>(ws + plan.items_rec);
    p.item_ml = reinterpret_cast<float2 *>(ws + plan.item_stats);
    p.logits = reinterpret_cast<float *>(ws + plan.logits);
    p.weights = cache.weights;
  }
  p.padded = plan.padded;

  CUtensorMap maps[3];
  if (!encode_pool(&maps[0], cache.k1, d, cache, cache.k1_strides, fp8, p.piece_rows) ||
      !encode_pool(&maps[1], cache.k2, d, cache, cache.k2_strides, fp8, p.piece_rows) ||
      !encode_pool(&maps[2], cache.v, 2 * d, cache, cache.v_strides, false, p.piece_rows))
    return DIFFATTN_ERR_CUDA;

  const bool two = plan.row_tiles == 2;
  diffattn_status st;
  if (d == 64)
    st = fp8 ? (two ? launch_main<64, true, 2>(p, maps, plan.ctas, stream)
                    : launch_main<64, true, 1>(p, maps, plan.ctas, stream))
             : (two ? launch_main<64, false, 2>(p, maps, plan.ctas, stream)
                    : launch_main<64, false, 1>(p, maps, plan.ctas, stream));
  else
    st = fp8 ? (two ? launch_main<128, true, 2>(p, maps, plan.ctas, stream)
                    : launch_main<128, true, 1>(p, maps, plan.ctas, stream))
             : (two ? launch_main<128, false, 2>(p, maps, plan.ctas, stream)
                    : launch_main<128, false, 1>(p, maps, plan.ctas, stream));
  if (st != DIFFATTN_OK) return st;
  JoinParams jp;
  jp.f = p;
  jp.ctas = plan.whole ? 1 : plan.ctas;
  jp.row_tile = 8 * plan.row_tiles;
  jp.join_rows = p.rows < jp.row_tile ? p.rows : jp.row_tile;
  jp.weight_chunks =
      accumulate ? static_cast<int32_t>((plan.padded + kWeightKeys - 1) / kWeightKeys) : 0;
  return d == 64 ? launch_join<64>(jp, stream) : launch_join<128>(jp, stream);
}

}  // namespace diffattn
