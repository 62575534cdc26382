// diffpaged_fwd: the plan, the launch and the second kernel (the main kernel is
// in paged_fwd.cuh).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "debug_check.cuh"
#include "paged.h"
#include "paged_fwd.cuh"
#include "ptx.cuh"

namespace diffattn {
namespace {

// The parts that the item whose steps begin at `start` is cut into: that of the CTA c0 with its
// first tile is in slot 2 c0 + 1 where its share begins before the item and in 2 c0 otherwise, the
// next ones' in 2 (c0 + 1), 2 (c0 + 2) ..
struct Parts {
  int32_t first, n;
  __device__ __forceinline__ int32_t slot(int32_t k) const {
    return k == 0 ? first : 2 * (first / 2 + k);
  }
};
__device__ __forceinline__ Parts parts_of(const Shares &all, uint32_t start, uint32_t units) {
  const uint32_t c0 = all.cta_of(start + kItemCost);
  return {static_cast<int32_t>(2 * c0 + (all.begin(c0) < start ? 1 : 0)),
          static_cast<int32_t>(all.cta_of(start + kItemCost + units - 1) - c0 + 1)};
}

// ---------------------------------------------------------------------------
// The second kernel: joins the items that a CTA boundary cut and adds the
// keys' weights.  Launched dependent on the first: it works out from kv_len
// what is cut where while that one runs, and then awaits its end.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;
constexpr int kMaxParts = 256;       // more than SMs
constexpr int kMaxRowBlocks = kPagedMaxTokens * kPagedMaxGroup / 32;
static_assert(kMaxRowBlocks <= 32, "a lane each");
constexpr int kWeightBlocks = 912;  // in all, about: two rounds of three per SM

constexpr size_t kDiscardBytes = size_t{16} << 20;

// Rows of a plane of the logits, by the rows of a block of the main kernel.
int plane_rows(int row_tile) { return row_tile < 4 ? row_tile : 4; }

struct JoinParams {
  FwdParams f;
  int32_t ctas, join_rows, row_tile;  // row_tile: rows of a block of the main kernel
  int32_t by_item;                    // joins are numbered by item, else by boundary
  uint32_t joins;                     // blocks that join
  int32_t weight_blocks;              // per (sequence, key/value head); 0 without weights
  int32_t row_groups;                 // warps that share a key's planes (1, 2, 4 or 8)
  // The logits are so many that L2 would write most of them out (8 x 8 x 32768 keys of four rows,
  // 67 MB: discarded once read, a call takes 200 us instead of 207); below, it costs 0.3 us.
  int32_t discard;
};

__device__ __forceinline__ void discard_line(void *line) {
  asm volatile("discard.global.L2 [%0], 128;" ::"l"(line) : "memory");
}

__device__ __forceinline__ bool timed_out(const FwdParams &p) {
  return p.status != nullptr &&
         *reinterpret_cast<volatile const int32_t *>(p.status) == DIFFATTN_ERR_TIMEOUT;
}

__device__ __forceinline__ float block_sum(float x, float *scratch) {
  x = warp_sum(x);
  if (threadIdx.x % 32 == 0) scratch[threadIdx.x / 32] = x;
  __syncthreads();
  float y = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) y += scratch[w];
  __syncthreads();
  return y;
}

// The shares, and the steps per head and row block before sequence b (one warp).
__device__ __forceinline__ Shares all_shares(const FwdParams &p, uint32_t ctas, int32_t b,
                                             uint32_t *before) {
  const int32_t most = p.max_pages * p.page_size;
  uint32_t total = 0, mine = 0, longest = 0, shortest = 0xFFFFFFFFu;
  for (int32_t x = threadIdx.x % 32; x < p.B; x += 32) {
    const uint32_t u = kItemCost + units_of(p.kv_len[x], most);
    total += u;
    mine += x < b ? u : 0;
    longest = max(longest, u);
    shortest = min(shortest, u);
  }
  *before = __reduce_add_sync(0xffffffffu, mine);
  return cut_line(p, __reduce_add_sync(0xffffffffu, total),
                  __reduce_max_sync(0xffffffffu, longest),
                  __reduce_min_sync(0xffffffffu, shortest), ctas);
}

// Block (cut item, row): joins one row.  The cut items are found from the boundaries between
// shares (each item by its first one) or, where these are fewer, from all items.
template <int kD>
__device__ void join_row(const JoinParams &jp) {
  const FwdParams &p = jp.f;
  __shared__ float factor[2][kMaxParts];
  __shared__ float scratch[kJoinThreads / 32];
  __shared__ float half[2 * kD];
  __shared__ int4 cut;  // item, its parts, the sequence's length; item -1: nothing to do
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t which = blockIdx.x / jp.join_rows;
  const int row = static_cast<int>(blockIdx.x - which * jp.join_rows);
  if (warp == 0) {
    int4 x = make_int4(-1, 0, 0, 0);
    Parts parts = {0, 1};
    if (jp.by_item) {
      const uint32_t bh = which / p.row_blocks;
      const int32_t b = static_cast<int32_t>(bh / p.kv_heads);
      uint32_t before;
      const Shares all = all_shares(p, jp.ctas, b, &before);
      const int32_t len = p.kv_len[b];
      const uint32_t units = units_of(len, p.max_pages * p.page_size);
      const uint32_t heads = p.kv_heads * p.row_blocks;
      if (all.mode == kPagedCut)
        parts = parts_of(all, before * heads + (which - b * heads) * (kItemCost + units), units);
      if (parts.n > 1) x = make_int4(static_cast<int>(which), parts.first, parts.n, len);
    } else {
      const Share s = find_share(p, which + 1, jp.ctas);
      if (s.all.mode == kPagedCut && s.off > kItemCost) {
        parts = parts_of(s.all, s.begin - s.off, s.units);
        if (parts.first / 2 == static_cast<int>(which))
          x = make_int4((s.b * p.kv_heads + s.hk) * p.row_blocks + s.rb, parts.first, parts.n,
                        s.len);
      }
    }
    if (lane == 0) cut = x;
  }
  __syncthreads();
  if (cut.x < 0 || cut.z > kMaxParts) return;
  const Parts parts = {cut.y, cut.z};
  const int32_t len = cut.w;
  const int rb = cut.x % p.row_blocks, bh = cut.x / p.row_blocks;
  const int hk = bh % p.kv_heads, b = bh / p.kv_heads;
  const int r = rb * jp.row_tile + row;
  if (r >= p.rows) return;
  const int i = p.by_group.div(r), h = hk * p.group + r - i * p.group;
  constexpr int kGroups = kJoinThreads / (2 * kD);  // threads per column: 2 (d = 64) or 1
  constexpr int kAhead = 4;
  const int col = threadIdx.x % (2 * kD), part = threadIdx.x / (2 * kD);
  const float *src = p.part + static_cast<int64_t>(row) * (2 * kD) + col;
  const int64_t map_step = static_cast<int64_t>(jp.row_tile) * (2 * kD);
  const float lam = __ldg(p.lambda + h);
  const float gain = p.headnorm && p.norm_w != nullptr ? __ldg(p.norm_w + h * (2 * kD) + col) : 1.f;
  grid_dependency_wait();

  // The first parts' values are on their way while the factors 2^(m_s - M) / l of both maps,
  // l = sum 2^(m_s - M) l_s, are formed by warps 0 and 1 (l_s < 0: a bad page or length).
  float ahead[kAhead][2];
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (part + kGroups * k < parts.n) {
      const float *x = src + parts.slot(part + kGroups * k) * 2 * map_step;
      ahead[k][0] = x[0];
      ahead[k][1] = x[map_step];
    }
  if (warp < 2) {
    float top = -INFINITY, sum = 0.f;
    bool bad = false;
    for (int k = lane; k < parts.n; k += 32)
      top = fmaxf(top, p.part_ml[(parts.slot(k) * 2ll + warp) * jp.row_tile + row].x);
    top = warp_max(top);
    for (int k = lane; k < parts.n; k += 32) {
      const float2 ml = p.part_ml[(parts.slot(k) * 2ll + warp) * jp.row_tile + row];
      const float f = ml.x == top ? 1.f : exp2f(ml.x - top);
      factor[warp][k] = f;
      sum += f * ml.y;
      bad |= ml.y < 0.f;
    }
    sum = warp_sum(sum);
    if (__any_sync(0xffffffffu, bad)) sum = NAN;
    const float c = (warp ? -lam : 1.f) / sum;
    for (int k = lane; k < parts.n; k += 32) factor[warp][k] *= c;
  }
  __syncthreads();
  float o = 0.f;
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (part + kGroups * k < parts.n)
      o = fmaf(factor[0][part + kGroups * k], ahead[k][0],
               fmaf(factor[1][part + kGroups * k], ahead[k][1], o));
#pragma unroll 4
  for (int k = part + kGroups * kAhead; k < parts.n; k += kGroups) {
    const float *x = src + parts.slot(k) * 2 * map_step;
    o = fmaf(factor[0][k], x[0], fmaf(factor[1][k], x[map_step], o));
  }
  if (kGroups == 2) {
    if (part == 1) half[col] = o;
    __syncthreads();
    if (part == 0) o += half[col];
  }
  const bool none = len - p.N + i < 0;  // padding: sees no key (the factors are not numbers)
  if (none || part != 0) o = 0.f;       // each column counted once
  if (p.headnorm == 2) {
    o -= block_sum(o, scratch) * (0.5f / kD);
    if (part != 0) o = 0.f;
  }
  if (p.headnorm) {
    const float ss = block_sum(o * o, scratch);
    if (!none) o *= rsqrtf(ss * (0.5f / kD) + p.eps) * p.out_scale * gain;
  }
  if (part == 0)
    p.out[b * p.outs.b + h * p.outs.h + i * p.outs.n + col] =
        __float2bfloat16_rn(timed_out(p) ? NAN : o);
}

template <int kN>
__device__ __forceinline__ void load_row(const float *src, float (&x)[kN]) {
  if constexpr (kN == 1) {
    x[0] = *src;
  } else if constexpr (kN == 2) {
    const float2 y = *reinterpret_cast<const float2 *>(src);
    x[0] = y.x, x[1] = y.y;
  } else {
    const float4 y = *reinterpret_cast<const float4 *>(src);
    x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w;
  }
}

// Block (sequence, key/value head, k): weights[j] += sum_r |map1 - lambda map2| of every
// weight_blocks-th run of keys.  A thread takes four keys of every row_groups-th plane of kPlane
// rows, both maps of a plane in flight; the groups' sums are added in their order.
//
// Bound: the logits (8 bytes a key and row, written by the main kernel and read here) go through L2
// at about 4 TB/s, and a call with few tiles waits for the rows' statistics.  8 x 8 x 32768 keys of
// four rows: 196 us where the call without weights takes 166, 20 us of it in the main kernel's
// stores; 5 x 4 rows, 4 x 4 heads of 300 to 3001 keys: 24.5 us, without weights 17.
template <int kPlane>
__device__ void add_weights(const JoinParams &jp, uint32_t block) {
  const FwdParams &p = jp.f;
  extern __shared__ float4 row_stat[];  // per row: M1, 1 / l1, M2, lambda / l2
  __shared__ float4 sums[kJoinThreads];
  __shared__ Parts item_parts[kMaxRowBlocks];
  __shared__ int shared_parts;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int groups = jp.row_groups, group = warp & (groups - 1);
  const int run = kJoinThreads * 4 / groups;  // keys of a pass
  const uint32_t bh = block / jp.weight_blocks;
  const int b = static_cast<int>(bh / p.kv_heads), hk = static_cast<int>(bh - b * p.kv_heads);
  const int32_t len = p.kv_len[b];
  const int32_t most = p.max_pages * p.page_size;
  const int32_t first = static_cast<int32_t>(block - bh * jp.weight_blocks) * run;
  if (len < 0 || len > most || first >= len) return;
  // While the main kernel runs: the parts of the item's row blocks, and the factors of the rows'
  // maps, 1 (0 for a row that sees no key and adds nothing) and lambda.
  if (warp == 0) {
    Parts parts = {0, 1};
    if (p.mode == kPagedByLengths) {
      uint32_t before;
      const Shares all = all_shares(p, jp.ctas, b, &before);
      const uint32_t units = units_of(len, most);
      if (all.mode == kPagedCut && lane < p.row_blocks)
        parts = parts_of(all,
                         before * p.kv_heads * p.row_blocks +
                             (hk * p.row_blocks + lane) * (kItemCost + units),
                         units);
    }
    if (lane < p.row_blocks) item_parts[lane] = parts;
    const int most_parts = __reduce_max_sync(0xffffffffu, parts.n);
    if (lane == 0) shared_parts = most_parts;
  }
  for (int r = threadIdx.x; r < p.rows; r += kJoinThreads) {
    const int i = p.by_group.div(r);
    const bool none = len - p.N + i < 0;
    row_stat[r] = make_float4(0.f, none ? 0.f : 1.f, 0.f,
                              __ldg(p.lambda + hk * p.group + r - i * p.group));
  }
  __syncthreads();
  int wide = 1;
  while (wide < 32 && wide < shared_parts) wide *= 2;
  const int own = lane & (wide - 1), per_round = kJoinThreads / wide;
  grid_dependency_wait();
  if (timed_out(p)) return;

  // A pass's first loads: the logits of this warp's first plane, and where the weights are.
  const int32_t *table = p.page_table + static_cast<int64_t>(b) * p.max_pages;
  float *logits = p.logits + static_cast<int64_t>(bh) * 2 * p.planes * p.padded * kPlane;
  const int64_t map_step = p.planes * p.padded * kPlane;
  int32_t key0 = first + (warp / groups) * 128;  // this warp's 128 keys
  float x1[4][kPlane], x2[4][kPlane];
  int32_t pages[4] = {0, 0, 0, 0};
  const auto load_plane = [&](int plane) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int32_t key = key0 + 32 * j + lane;
      if (key < len && plane < p.planes) {
        const float *src = logits + (plane * p.padded + key) * kPlane;
        load_row(src, x1[j]);
        load_row(src + map_step, x2[j]);
      }
    }
  };
  const auto load_pass = [&] {
    load_plane(group);
    if (group == 0)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int32_t key = key0 + 32 * j + lane;
        if (key < len) pages[j] = __ldg(table + p.by_page.div(key));
      }
  };
  load_pass();

  // The rows' statistics: `wide` lanes per row and map, up to four of them in flight.
  const auto part_state = [&](int k, int part) {  // row k / 2, map k % 2
    const int r = k >> 1, rb = r / jp.row_tile;
    const Parts parts = item_parts[rb];
    if (part >= parts.n) return make_float2(-INFINITY, 0.f);
    const int64_t at =
        parts.n == 1 ? static_cast<int64_t>(bh) * p.row_blocks + rb : parts.slot(part);
    return (parts.n == 1 ? p.item_ml
                         : p.part_ml)[(at * 2 + (k & 1)) * jp.row_tile + r - rb * jp.row_tile];
  };
  bool bad = false;
#pragma unroll 1
  for (int k0 = 0; k0 < 2 * p.rows; k0 += 4 * per_round) {
    float2 ml[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = k0 + j * per_round + threadIdx.x / wide;
      ml[j] = k < 2 * p.rows ? part_state(k, own) : make_float2(-INFINITY, 0.f);
      bad |= ml[j].y < 0.f;
    }
    if (shared_parts > 32)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + j * per_round + threadIdx.x / wide;
        if (k < 2 * p.rows)
#pragma unroll 1
          for (int s = own + 32; s < shared_parts; s += 32) {
            const float2 more = part_state(k, s);
            bad |= more.y < 0.f;
            const float y = fmaxf(ml[j].x, more.x);
            ml[j].y = (ml[j].x == y ? ml[j].y : ml[j].y * ex2_approx(ml[j].x - y)) +
                      (more.x == y ? more.y : ex2_approx(more.x - y) * more.y);
            ml[j].x = y;
          }
      }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (k0 + j * per_round >= 2 * p.rows) break;
      const int k = k0 + j * per_round + threadIdx.x / wide;
      float y = ml[j].x;
      for (int o = wide / 2; o > 0; o >>= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o));
      float sum = ml[j].x == y ? ml[j].y : ml[j].y * ex2_approx(ml[j].x - y);
      for (int o = wide / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (own == 0 && k < 2 * p.rows) {
        float *out = reinterpret_cast<float *>(row_stat + (k >> 1)) + 2 * (k & 1);
        out[0] = y;
        out[1] = (k & 1) == 0 && out[1] == 0.f ? 0.f : __fdividef(out[1], sum);
      }
    }
  }
  if (__syncthreads_or(bad)) return;  // a bad page: the sequence's weights stay as they are
#pragma unroll 1
  for (int32_t at = first; at < len; at += run * jp.weight_blocks) {
    float *to[4];
    float old[4], w[4] = {0.f, 0.f, 0.f, 0.f};
    if (group == 0)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int32_t key = key0 + 32 * j + lane;
        to[j] = p.weights + p.by_page.mod(key) +
                (static_cast<int64_t>(pages[j]) * p.kv_heads + hk) * p.page_size;
        if (key < len) old[j] = *to[j];
      }
#pragma unroll 1
    for (int plane = group; plane < p.planes; plane += groups) {
      if (plane != group) load_plane(plane);
#pragma unroll
      for (int e = 0; e < kPlane; ++e) {
        const int r = plane * kPlane + e;
        if (r >= p.rows) break;
        const float4 st = row_stat[r];
        if (st.y == 0.f) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] += fabsf(ex2_approx(x1[j][e] - st.x) * st.y - ex2_approx(x2[j][e] - st.z) * st.w);
      }
      // The logits are not needed any more: many of them are dropped before L2 writes them out.
      if (jp.discard) {
        __syncwarp();
        constexpr int kLines = 4 * kPlane;  // of 128 keys of a plane and map
        if (lane < 2 * kLines && key0 < len)
          discard_line(logits + (plane * p.padded + key0) * kPlane + (lane / kLines) * map_step +
                       lane % kLines * 32);
      }
    }
    const int32_t here = key0 + lane;
    key0 += run * jp.weight_blocks;
    if (at + run * jp.weight_blocks < len) load_pass();
    if (groups > 1) {
      sums[threadIdx.x] = make_float4(w[0], w[1], w[2], w[3]);
      __syncthreads();
      if (group == 0)
        for (int k = 1; k < groups; ++k) {
          const float4 y = sums[threadIdx.x + 32 * k];
          w[0] += y.x;
          w[1] += y.y;
          w[2] += y.z;
          w[3] += y.w;
        }
      __syncthreads();
    }
    if (group == 0)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (here + 32 * j < len) *to[j] = old[j] + w[j];
  }
}

// kPlane: rows of a plane of the logits; 0 where no weights are added.
template <int kD, int kPlane>
__global__ void __launch_bounds__(kJoinThreads, kPlane ? 3 : 6)
    diffpaged_join_kernel(const __grid_constant__ JoinParams jp) {
  if (kPlane == 0 || blockIdx.x < jp.joins) {
    join_row<kD>(jp);
  } else {
    if constexpr (kPlane > 0) add_weights<kPlane>(jp, blockIdx.x - jp.joins);
  }
  // Blocks with nothing to do leave, but for the first: were there no others (no item cut), this
  // kernel would end, and the one behind it on the stream begin, before the main kernel has.
  if (blockIdx.x == 0) grid_dependency_wait();
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

template <int kD, int kPlane>
diffattn_status launch_join_of(const JoinParams &jp, cudaStream_t stream) {
  const int64_t blocks = static_cast<int64_t>(jp.joins) +
                         static_cast<int64_t>(jp.f.B) * jp.f.kv_heads * jp.weight_blocks;
  if (blocks == 0) return DIFFATTN_OK;
  if (blocks > INT32_MAX) return DIFFATTN_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = jp.weight_blocks ? sizeof(float4) * jp.f.rows : 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, diffpaged_join_kernel<kD, kPlane>, jp) == cudaSuccess
             ? DIFFATTN_OK
             : DIFFATTN_ERR_CUDA;
}

template <int kD>
diffattn_status launch_join(const JoinParams &jp, cudaStream_t stream) {
  const int plane = jp.weight_blocks ? plane_rows(jp.row_tile) : 0;
  return plane == 0   ? launch_join_of<kD, 0>(jp, stream)
         : plane == 1   ? launch_join_of<kD, 1>(jp, stream)
         : plane == 2 ? launch_join_of<kD, 2>(jp, stream)
                      : launch_join_of<kD, 4>(jp, stream);
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

bool plan_paged_fwd(const diffattn_desc &desc, const diffpaged_cache &cache, bool accumulate,
                    int sm_count, PagedFwdPlan *plan) {
  PagedFwdPlan &q = *plan;
  q = PagedFwdPlan{};
  const int64_t rows = desc.N * (desc.H / cache.kv_heads);
  q.row_tile = 1;
  while (q.row_tile < rows && q.row_tile < 32) q.row_tile *= 2;
  const int64_t row_tile = q.row_tile;
  q.row_blocks = static_cast<int>((rows + row_tile - 1) / row_tile);
  const double items =
      static_cast<double>(desc.B) * static_cast<double>(cache.kv_heads) * q.row_blocks;
  if (items > INT32_MAX) return false;
  q.items = desc.B * cache.kv_heads * q.row_blocks;
  const int64_t most = cache.max_pages * cache.page_size;
  const int64_t units = (most + kTile - 1) / kTile;
  q.padded = units * kTile;
  if (items * static_cast<double>(units + kItemCost) >= 2147483648.0) return false;
  // The kernels choose from the lengths how items are taken (cut_line).  Where the choice is the
  // same for all lengths up to the capacity, it is made here, and the second kernel and its
  // workspace are left out: one CTA per item where that is right for full sequences and, as the
  // launch is saved too, costs at most kSecondKernel tiles more where only one sequence is full; an
  // uncut share is longest - 1 steps longer at most, and where all items are equally long, as those
  // of a single sequence are, `per` of them long.
  const int64_t heads = cache.kv_heads * q.row_blocks;
  const int64_t per = (q.items + sm_count - 1) / sm_count;
  const int64_t alone = int64_t{kMostAlone} * sm_count, uneven = int64_t{kUneven} * sm_count;
  q.mode = kPagedByLengths;
  if (q.items <= sm_count) {
    if (units * (sm_count - q.items) <= alone &&
        units * (sm_count - heads) - (q.items - heads) <= alone + kSecondKernel * sm_count)
      q.mode = kPagedWhole;
  } else if (units + kItemCost <= kUneven ||
             (desc.B == 1 && (units + kItemCost) * (per * sm_count - q.items) <= uneven)) {
    q.mode = kPagedUncut;
  }
  q.ctas = q.mode == kPagedWhole ? static_cast<int>(q.items) : sm_count;
  if (q.items * (units + kItemCost) < q.ctas)
    q.ctas = static_cast<int>(q.items * (units + kItemCost));
  const size_t slots = q.mode == kPagedByLengths ? 2 * static_cast<size_t>(q.ctas) : 0;
  size_t at = 0;
  const auto take = [&at](size_t bytes) {
    const size_t here = at;
    at += round256(bytes);
    return here;
  };
  q.part = take(slots * 2 * row_tile * 2 * desc.d * sizeof(float));
  q.stats = take(slots * 2 * row_tile * sizeof(float2));
  if (accumulate) {
    const int64_t plane = plane_rows(q.row_tile), kept = (rows + plane - 1) / plane * plane;
    const double logits = static_cast<double>(desc.B) * static_cast<double>(cache.kv_heads) * 2.0 *
                          static_cast<double>(kept) * static_cast<double>(q.padded) * 4.0;
    if (logits > 1.0e18) return false;
    q.item_stats = take(q.items * 2 * row_tile * sizeof(float2));
    q.logits = take(static_cast<size_t>(desc.B * cache.kv_heads * 2 * kept * q.padded) *
                    sizeof(float));
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
  p.by_page = fast_div(static_cast<uint32_t>(p.page_size));
  p.by_group = fast_div(static_cast<uint32_t>(p.group));
  p.causal = desc.causal ? 1 : 0;
  p.headnorm = desc.headnorm;
  p.mode = plan.mode;
  p.eps = desc.eps;
  p.out_scale = 1.0f - desc.lambda_init;
  p.scale_log2 = kLog2e / std::sqrt(static_cast<float>(d));
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  if (plan.mode == kPagedByLengths) {
    p.part = reinterpret_cast<float *>(ws + plan.part);
    p.part_ml = reinterpret_cast<float2 *>(ws + plan.stats);
  }
  if (accumulate) {
    p.item_ml = reinterpret_cast<float2 *>(ws + plan.item_stats);
    p.logits = reinterpret_cast<float *>(ws + plan.logits);
    p.weights = cache.weights;
    p.planes = (p.rows + plane_rows(plan.row_tile) - 1) / plane_rows(plan.row_tile);
  }
  p.padded = plan.padded;

  CUtensorMap maps[3];
  if (!encode_pool(&maps[0], cache.k1, d, cache, cache.k1_strides, fp8, p.piece_rows) ||
      !encode_pool(&maps[1], cache.k2, d, cache, cache.k2_strides, fp8, p.piece_rows) ||
      !encode_pool(&maps[2], cache.v, 2 * d, cache, cache.v_strides, false, p.piece_rows))
    return DIFFATTN_ERR_CUDA;

  const diffattn_status st = d == 64 ? launch_paged_main_d64(p, maps, plan, fp8, stream)
                                     : launch_paged_main_d128(p, maps, plan, fp8, stream);
  if (st != DIFFATTN_OK) return st;
  JoinParams jp = {};
  jp.f = p;
  jp.ctas = plan.ctas;
  jp.row_tile = plan.row_tile;
  jp.join_rows = p.rows < jp.row_tile ? p.rows : jp.row_tile;
  // Cut items are at most one per boundary.
  const int64_t cuts = plan.mode == kPagedByLengths ? plan.ctas - 1 : 0;
  jp.by_item = plan.items < cuts ? 1 : 0;
  jp.joins = static_cast<uint32_t>((jp.by_item ? plan.items : cuts) * jp.join_rows);
  jp.discard = plan.bytes - plan.logits >= kDiscardBytes ? 1 : 0;
  if (accumulate) {
    // As many blocks as find work, but not more than a few per SM, as each forms the rows'
    // statistics.  Planes go to warps of their own while that makes more blocks than would wait.
    const int64_t heads = desc.B * cache.kv_heads;
    const int64_t share = (int64_t{kWeightBlocks} + heads - 1) / heads;
    const auto runs = [&] {
      const int64_t run = 4 * kJoinThreads / jp.row_groups;
      return (plan.padded + run - 1) / run;
    };
    jp.row_groups = 1;
    while (jp.row_groups < 8 && jp.row_groups < p.planes && runs() < share) jp.row_groups *= 2;
    jp.weight_blocks = static_cast<int32_t>(runs() < share ? runs() : share);
  }
  return d == 64 ? launch_join<64>(jp, stream) : launch_join<128>(jp, stream);
}

}  // namespace diffattn
