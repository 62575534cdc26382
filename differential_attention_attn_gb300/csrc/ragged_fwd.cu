// diffragged_fwd: the plan, the launches and the second kernel, which joins the
// items that a border between shares cut (the main kernels are in
// ragged_fwd_d64.cu and ragged_fwd_d128.cu).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "debug_check.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "ragged_fwd.cuh"

namespace diffattn {
namespace {

// Block (share, 32 rows) joins the item that share begins and others go on with: a row a lane, 8
// or 16 columns a warp, so that every read of a part is a whole line.  Latency bounds it (a few
// parts of each item): all values of two parts are on their way at a time.
constexpr int kJoinWarps = 16;
template <int DV>
__global__ void __launch_bounds__(32 * kJoinWarps)
    diffragged_join_kernel(const __grid_constant__ RaggedParams p) {
  constexpr int kWarps = kJoinWarps, kCols = DV / kWarps;
  __shared__ float sums[kWarps][33];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  grid_dependency_wait();
  const RaggedJoin j = p.joins[blockIdx.x];
  grid_dependents_launch();
  const int r = blockIdx.y * 32 + lane, rows = j.tokens * p.group;
  if (j.parts <= 0 || static_cast<int>(blockIdx.y) * 32 >= rows) return;
  constexpr int64_t kMap = part_floats(DV);
  const auto part = [&](int k) {
    return p.part + (k == 0 ? j.slot : 2ll * (j.slot / 2 + k)) * 2 * kMap + r;
  };
  const int32_t token = p.by_group.div(r), h = j.hk * p.group + r - token * p.group;
  const bool mine = r < rows;
  const float lam = mine ? p.lambda[h] : 0.f;
  float gain[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i)
    gain[i] = p.headnorm && p.norm_w != nullptr && mine ? p.norm_w[h * DV + kCols * warp + i] : 1.f;
  // Against the largest reference so far, as the parts were against theirs.
  float top[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[2][kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i) o[0][i] = o[1][i] = 0.f;
#pragma unroll 2
  for (int k = 0; k < j.parts; ++k) {
    const float *src = part(k);
    float x[2][kCols], ref[2], sum[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      ref[m] = src[m * kMap + DV * kTile];
      sum[m] = src[m * kMap + (DV + 1) * kTile];
#pragma unroll
      for (int i = 0; i < kCols; ++i) x[m][i] = src[m * kMap + (kCols * warp + i) * kTile];
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const float now = fmaxf(top[m], ref[m]);
      const float old = top[m] == now ? 1.f : exp2f(top[m] - now);
      const float f = ref[m] == now ? 1.f : exp2f(ref[m] - now);
      top[m] = now;
      l[m] = l[m] * old + f * sum[m];
#pragma unroll
      for (int i = 0; i < kCols; ++i) o[m][i] = o[m][i] * old + f * x[m][i];
    }
  }
  const float c1 = 1.f / l[0], c2 = lam / l[1];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < kCols; ++i) {
    o[0][i] = o[0][i] * c1 - o[1][i] * c2;
    ss = fmaf(o[0][i], o[0][i], ss);
  }
  if (p.headnorm) {
    const auto over_row = [&](float x) {
      sums[warp][lane] = x;
      __syncthreads();
      float y = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) y += sums[w][lane];
      __syncthreads();
      return y;
    };
    if (p.headnorm == 2) {
      float sm = 0.f;
#pragma unroll
      for (int i = 0; i < kCols; ++i) sm += o[0][i];
      const float mu = over_row(sm) * (1.f / DV);
      ss = 0.f;
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        o[0][i] -= mu;
        ss = fmaf(o[0][i], o[0][i], ss);
      }
    }
    const float rr = rsqrtf(over_row(ss) * (1.f / DV) + p.eps) * p.out_scale;
#pragma unroll
    for (int i = 0; i < kCols; ++i) o[0][i] *= rr * gain[i];
  }
  if (!mine) return;
  if (j.first + token < 0) {
#pragma unroll
    for (int i = 0; i < kCols; ++i) o[0][i] = 0.f;
  }
  if (!dbg_ok(j.row + token < p.N, p.status, 110)) return;
  uint4 *out =
      reinterpret_cast<uint4 *>(p.out + (j.row + token) * p.out_n + h * p.out_h + kCols * warp);
#pragma unroll
  for (int i = 0; i < kCols; i += 8)
    out[i / 8] = make_uint4(pack_bf16x2(o[0][i], o[0][i + 1]), pack_bf16x2(o[0][i + 2], o[0][i + 3]),
                            pack_bf16x2(o[0][i + 4], o[0][i + 5]),
                            pack_bf16x2(o[0][i + 6], o[0][i + 7]));
}

template <int DV>
cudaError_t launch_join(const RaggedParams &p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.shares), 4);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, diffragged_join_kernel<DV>, p);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled_fn() {
  static EncodeTiledFn fn = [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<EncodeTiledFn>(ptr);
  }();
  return fn;
}

// A tensor map of `rank` dimensions, the innermost contiguous, in boxes at most 128 bytes wide.
bool encode(CUtensorMap *map, const void *base, int rank, const cuuint64_t *dims,
            const int64_t *strides, const cuuint32_t *box, bool fp8) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (fn == nullptr) return false;
  const cuuint64_t es = fp8 ? 1 : 2;
  cuuint64_t bytes[3];
  for (int i = 0; i + 1 < rank; ++i) bytes[i] = static_cast<cuuint64_t>(strides[i]) * es;
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return fn(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
            const_cast<void *>(base), dims, bytes, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
            box[0] * es == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
cuuint32_t box_width(int64_t width, bool fp8) {
  const int64_t most = fp8 ? 128 : 64;
  return static_cast<cuuint32_t>(width < most ? width : most);
}
// Packed rows {width, heads, tokens}: a group of heads of `tokens` tokens.
bool encode_packed(CUtensorMap *map, const void *base, int64_t width, int64_t heads, int64_t rows,
                   const diffattn_strides &st, bool fp8, int group, int tokens) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(rows)};
  const int64_t strides[2] = {st.h, st.n};
  const cuuint32_t box[3] = {box_width(width, fp8), static_cast<cuuint32_t>(group),
                             static_cast<cuuint32_t>(tokens)};
  return encode(map, base, 3, dims, strides, box, fp8);
}
// A pool {width, page_size, heads, pages}: `rows` rows of a page.
bool encode_pool(CUtensorMap *map, const void *base, int64_t width, const diffpaged_cache &c,
                 const diffattn_strides &st, bool fp8, int rows) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(c.page_size),
                              static_cast<cuuint64_t>(c.kv_heads),
                              static_cast<cuuint64_t>(c.num_pages)};
  const int64_t strides[3] = {st.n, st.h, st.b};
  const cuuint32_t box[4] = {box_width(width, fp8), static_cast<cuuint32_t>(rows), 1, 1};
  return encode(map, base, 4, dims, strides, box, fp8);
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

bool plan_ragged_fwd(const diffattn_desc &desc, const diffpaged_cache &cache, int sm_count,
                     RaggedFwdPlan *plan) {
  RaggedFwdPlan &q = *plan;
  q = RaggedFwdPlan{};
  q.shares = desc.d == 64 ? sm_count : sm_count / 2;
  // Items this short are never cut (cut_line).
  const int64_t units = (cache.max_pages * cache.page_size + kTile - 1) / kTile;
  // A line has fewer than 2^31 steps, however full the batch and the table.
  const int64_t tokens = kTile / (desc.H / cache.kv_heads);
  if (static_cast<double>(cache.kv_heads) * static_cast<double>(desc.N / tokens + desc.B) *
          static_cast<double>(kItemSteps + units * kTileSteps) >=
      2147483648.0)
    return false;
  q.joins = kItemSteps + units * kTileSteps > kJoinSteps;
  size_t at = 0;
  const auto take = [&at](size_t bytes) {
    const size_t here = at;
    at += round256(bytes);
    return here;
  };
  if (q.joins) {
    q.part = take(size_t{2} * q.shares * 2 * part_floats(2 * desc.d) * sizeof(float));
    q.join = take(q.shares * sizeof(RaggedJoin));
  }
  if (desc.d == 128) q.swap = take(ragged_swap_bytes(q.shares));
  q.bytes = at;
  return true;
}

diffattn_status launch_ragged_fwd(const diffattn_desc &desc, const diffpaged_cache &cache,
                                  const RaggedFwdPlan &plan, const int32_t *q_start, const void *q1,
                                  const void *q2, const float *lambda, const float *norm_w,
                                  void *out, const diffattn_strides strides[3], void *workspace,
                                  cudaStream_t stream) {
  const bool fp8 = desc.dtype == DIFFATTN_E4M3_QK;
  const int64_t d = desc.d;
  RaggedParams p = {};
  p.q_start = q_start;
  p.kv_len = cache.kv_len;
  p.page_table = cache.page_table;
  p.lambda = lambda;
  p.norm_w = norm_w;
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.status = desc.status_dev;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  if (plan.joins) {
    p.part = reinterpret_cast<float *>(ws + plan.part);
    p.joins = reinterpret_cast<RaggedJoin *>(ws + plan.join);
  }
  if (d == 128) p.swap = reinterpret_cast<float *>(ws + plan.swap);
  p.out_n = strides[2].n;
  p.out_h = strides[2].h;
  p.B = static_cast<int32_t>(desc.B);
  p.N = static_cast<int32_t>(desc.N);
  p.kv_heads = static_cast<int32_t>(cache.kv_heads);
  p.group = static_cast<int32_t>(desc.H / cache.kv_heads);
  p.tokens = kTile / p.group;
  p.group_bits = -1;
  for (int k = 0; k <= 6; ++k)
    if (p.group == 1 << k) p.group_bits = k;
  p.num_pages = static_cast<int32_t>(cache.num_pages);
  p.max_pages = static_cast<int32_t>(cache.max_pages);
  p.page_size = cache.page_size;
  p.piece_rows = 16;
  while (p.piece_rows < kTile && cache.page_size % (2 * p.piece_rows) == 0) p.piece_rows *= 2;
  p.causal = desc.causal ? 1 : 0;
  p.headnorm = desc.headnorm;
  p.shares = plan.shares;
  p.by_page = fast_div(static_cast<uint32_t>(p.page_size));
  p.by_group = fast_div(static_cast<uint32_t>(p.group));
  p.by_tokens = fast_div(static_cast<uint32_t>(p.tokens));
  p.eps = desc.eps;
  p.out_scale = 1.0f - desc.lambda_init;
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(d)));

  CUtensorMap maps[5];
  if (!encode_packed(&maps[0], q1, d, desc.H, desc.N, strides[0], fp8, p.group, p.tokens) ||
      !encode_packed(&maps[1], q2, d, desc.H, desc.N, strides[1], fp8, p.group, p.tokens) ||
      !encode_pool(&maps[2], cache.k1, d, cache, cache.k1_strides, fp8, p.piece_rows) ||
      !encode_pool(&maps[3], cache.k2, d, cache, cache.k2_strides, fp8, p.piece_rows) ||
      !encode_pool(&maps[4], cache.v, 2 * d, cache, cache.v_strides, false, p.piece_rows))
    return DIFFATTN_ERR_CUDA;
  const diffattn_status st = d == 64 ? launch_ragged_main_d64(p, maps, fp8, stream)
                                     : launch_ragged_main_d128(p, maps, fp8, stream);
  if (st != DIFFATTN_OK || !plan.joins) return st;
  const cudaError_t e = d == 64 ? launch_join<128>(p, stream) : launch_join<256>(p, stream);
  return e == cudaSuccess ? DIFFATTN_OK : DIFFATTN_ERR_CUDA;
}

}  // namespace diffattn
