// diffpaged_append: the newest tokens' k1, k2 and v rows into the pages of a
// cache.
//
// Token i of sequence b goes to position t = kv_len[b] - N + i (t < 0 is
// padding and is skipped): row t % page_size of page table[b][t / page_size].
// With an e4m3 key cache k1 and k2 are rounded on the way: to nearest, ties to
// even, saturating at +-448 (one conversion from the exact bf16 value; the
// attention then uses the stored values exactly).
//
// Bound: a copy, so HBM bandwidth for prompts (B Hkv N rows of 8 d bytes read
// and written) and the chain length -> page number -> store for a few tokens.
// A row of k1 | k2 | v is 32 (d = 64) or 64 sixteen-byte units, so each lane of
// a warp moves one or two of them (e4m3 keys leave as eight bytes each) and
// every access fills its sectors.
// Measured on GB300: 131072 rows at d = 64 (135 MB) 26.1 us, 76 % of the copy
// rate; 65536 rows at d = 128 22 us, 90 %; one token of 64 x 16 heads 1.9 us.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "debug_check.cuh"
#include "paged.h"
#include "ptx.cuh"

namespace diffattn {
namespace {

constexpr int kWarps = 8;
// Up to this many rows a warp takes one.  One / two rows a warp, us: 8192 rows at d = 64 3.2 / 3.9,
// 16384 4.7 / 4.7 (d = 128 5.9 / 6.0, e4m3 4.7 / 5.0), 32768 8.4 / 8.3 (with padding 7.2 / 6.5).
constexpr uint32_t kFewRows = 16384;

struct AppendParams {
  const uint8_t *src[3];  // k1, k2, v (bf16)
  uint8_t *dst[3];        // the pools
  int64_t src_b[3], src_h[3], src_n[3];  // strides in bytes
  int64_t dst_p[3], dst_h[3], dst_n[3];
  float *weights;
  const int32_t *page_table;
  const int32_t *kv_len;
  int32_t *status;
  uint32_t rows, groups;  // B * kv_heads * N; the warps that take them
  uint32_t N, kv_heads, page_size, max_pages, num_pages;
  FastDiv by_n, by_heads, by_page;
};

// Eight bf16 values as eight e4m3 values.
__device__ __forceinline__ uint2 to_e4m3(const uint4 &a) {
  const uint32_t in[4] = {a.x, a.y, a.z, a.w};
  uint32_t half[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = __uint_as_float(in[i] << 16), hi = __uint_as_float(in[i] & 0xFFFF0000u);
    half[i] = __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(half[0] | (half[1] << 16), half[2] | (half[3] << 16));
}

// A warp per kRows consecutive rows of a head.  kEager: loaded while their place is looked up, the
// shortest chain for a few new tokens; otherwise only once they are known to be no padding, which
// costs a prompt without padding less than eager loads cost one of which half is padding (65568
// rows of e4m3 keys at d = 128: 13.3 us, eager 21.4).  Two rows a warp: 131072 rows at d = 64 26.1
// us, one 27.2; e4m3 keys 26.6 and 28.5 us, four rows 25.2 (but 13.5 us in the case above).
template <int kD, bool kFp8, int kRows, bool kEager>
__global__ void __launch_bounds__(kWarps * 32, kRows == 1 ? 8 : 6)
    diffpaged_append_kernel(const AppendParams p) {
  constexpr int kKeyUnits = kD / 8;  // 16-byte units of a key row
  constexpr int kPerLane = (2 * kKeyUnits + kD / 4) / 32;
  static_assert(kPerLane * 32 == 2 * kKeyUnits + kD / 4, "no idle lanes");
  const int lane = threadIdx.x % 32;
  const uint32_t group = blockIdx.x * kWarps + threadIdx.x / 32;
  if (group >= p.groups) return;
  const uint32_t bh = p.by_n.div(group), i0 = (group - bh * p.by_n.d) * kRows;
  const uint32_t b = p.by_heads.div(bh), h = bh - b * p.kv_heads;
  grid_dependency_wait();
  grid_dependents_launch();
  const int32_t len = p.kv_len[b];

  uint4 x[kRows][kPerLane];
  int32_t page[kRows];
  const auto load = [&](int r) {
#pragma unroll
    for (int u = 0; u < kPerLane; ++u) {
      const int unit = lane + 32 * u;
      const int t = unit < kKeyUnits ? 0 : unit < 2 * kKeyUnits ? 1 : 2;
      const uint8_t *s = p.src[t] + b * p.src_b[t] + h * p.src_h[t] + (i0 + r) * p.src_n[t] +
                         (unit - t * kKeyUnits) * 16;
      // (A plain load: the rows may be the output of a kernel that this one has started under.)
      x[r][u] = *reinterpret_cast<const uint4 *>(s);
    }
  };
  if (kEager)
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (i0 + r < p.N) load(r);
  if (len < 0 || static_cast<uint32_t>(len) > p.max_pages * p.page_size) {
    report_bad_page(p.status);
    return;
  }
  const int32_t t0 = len - static_cast<int32_t>(p.N) + static_cast<int32_t>(i0);
  const auto wanted = [&](int r) { return i0 + r < p.N && t0 + r >= 0; };
#pragma unroll
  for (int r = 0; r < kRows; ++r)
    if (wanted(r)) {
      page[r] = __ldg(p.page_table + static_cast<int64_t>(b) * p.max_pages + p.by_page.div(t0 + r));
      if (!kEager) load(r);
    }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (!wanted(r)) continue;
    if (static_cast<uint32_t>(page[r]) >= p.num_pages) {
      report_bad_page(p.status);
      continue;
    }
    const int32_t slot = p.by_page.mod(t0 + r);
    if (!dbg_ok(slot >= 0 && static_cast<uint32_t>(slot) < p.page_size, p.status, 40)) continue;
#pragma unroll
    for (int u = 0; u < kPerLane; ++u) {
      const int unit = lane + 32 * u;
      const int t = unit < kKeyUnits ? 0 : unit < 2 * kKeyUnits ? 1 : 2;
      uint8_t *row = p.dst[t] + page[r] * p.dst_p[t] + h * p.dst_h[t] + slot * p.dst_n[t];
      const int off = unit - t * kKeyUnits;
      if (kFp8 && t < 2)
        reinterpret_cast<uint2 *>(row)[off] = to_e4m3(x[r][u]);
      else
        reinterpret_cast<uint4 *>(row)[off] = x[r][u];
    }
    if (lane == 0 && p.weights != nullptr)
      p.weights[(static_cast<int64_t>(page[r]) * p.kv_heads + h) * p.page_size + slot] = 0.f;
  }
}

template <int kD, bool kFp8, int kRows, bool kEager>
cudaError_t launch_rows(AppendParams p, cudaStream_t stream) {
  const uint32_t per_head = (p.N + kRows - 1) / kRows;
  p.by_n = fast_div(per_head);
  p.groups = p.rows / p.N * per_head;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.groups + kWarps - 1) / kWarps);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, diffpaged_append_kernel<kD, kFp8, kRows, kEager>, p);
}

template <int kD, bool kFp8>
cudaError_t launch(const AppendParams &p, cudaStream_t stream) {
  return p.rows <= kFewRows ? launch_rows<kD, kFp8, 1, true>(p, stream)
                            : launch_rows<kD, kFp8, 2, false>(p, stream);
}

}  // namespace

diffattn_status launch_paged_append(const diffattn_desc &desc, const diffpaged_cache &cache,
                                    const void *k1, const void *k2, const void *v,
                                    const diffattn_strides *strides, cudaStream_t stream) {
  const double rows = static_cast<double>(desc.B) * static_cast<double>(cache.kv_heads) *
                      static_cast<double>(desc.N);
  if (rows >= 2147483648.0) return DIFFATTN_ERR_UNSUPPORTED;  // a terabyte of rows
  const bool fp8 = desc.dtype == DIFFATTN_E4M3_QK;
  AppendParams p = {};
  const void *src[3] = {k1, k2, v};
  void *dst[3] = {cache.k1, cache.k2, cache.v};
  const diffattn_strides *ds[3] = {&cache.k1_strides, &cache.k2_strides, &cache.v_strides};
  for (int t = 0; t < 3; ++t) {
    const int64_t width = t == 2 ? 2 * desc.d : desc.d;
    const diffattn_strides s =
        strides ? strides[t]
                : diffattn_strides{cache.kv_heads * desc.N * width, desc.N * width, width};
    const int64_t es = (fp8 && t < 2) ? 1 : 2;
    p.src[t] = static_cast<const uint8_t *>(src[t]);
    p.dst[t] = static_cast<uint8_t *>(dst[t]);
    p.src_b[t] = 2 * s.b;
    p.src_h[t] = 2 * s.h;
    p.src_n[t] = 2 * s.n;
    p.dst_p[t] = es * ds[t]->b;
    p.dst_h[t] = es * ds[t]->h;
    p.dst_n[t] = es * ds[t]->n;
  }
  p.weights = cache.weights;
  p.page_table = cache.page_table;
  p.kv_len = cache.kv_len;
  p.status = desc.status_dev;
  p.rows = static_cast<uint32_t>(rows);
  p.N = static_cast<uint32_t>(desc.N);
  p.kv_heads = static_cast<uint32_t>(cache.kv_heads);
  p.page_size = static_cast<uint32_t>(cache.page_size);
  p.max_pages = static_cast<uint32_t>(cache.max_pages);
  p.num_pages = static_cast<uint32_t>(cache.num_pages);
  p.by_heads = fast_div(p.kv_heads);
  p.by_page = fast_div(p.page_size);
  cudaError_t e;
  if (desc.d == 64)
    e = fp8 ? launch<64, true>(p, stream) : launch<64, false>(p, stream);
  else
    e = fp8 ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
  return e == cudaSuccess ? DIFFATTN_OK : DIFFATTN_ERR_CUDA;
}

}  // namespace diffattn
