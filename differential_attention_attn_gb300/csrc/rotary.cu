// diffrotary_frequencies and diffrotary_apply (include/diffattn_rotary.h).
//
// Bound: a read and a write of every row, so HBM bandwidth.  A thread works out
// the eight cosines and sines of its (token, unit) once, from the 64-bit
// fractions, and takes kRows heads with them, whose loads are all on their way
// before the first is turned.  Measured on GB300: q1, q2, k1, k2 of 2 x 16 heads x
// 4096 tokens at d = 64, 134 MB: 19.8 us, the copy rate; d = 128, half of it turned
// back in neighbours, as much: 20.3 us; 48 tokens of 32 heads over 8: 2.0 us.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "debug_check.cuh"
#include "internal.h"
#include "paged.h"
#include "ptx.cuh"
#include "rotary.cuh"

namespace diffattn {
namespace {

constexpr int kThreads = 256;

struct RotaryTensor {
  const uint8_t *x;
  uint8_t *y;
  int64_t xb, xh, xn, yb, yh, yn;  // byte strides
  int32_t heads, slices;           // slices of kRows heads
};

struct RotaryParams {
  RotaryTensor t[4];
  const uint64_t *freq;
  const int32_t *positions;
  int64_t position_stride, start;
  uint32_t tokens, N;  // B * N, N
  int32_t unit_bits, rot;  // 2^unit_bits units in a row
  bool inverse;
  float scale;
  int32_t *status;
};

// Thread (token, unit) x block row (tensor, kRows heads of it).
template <typename T, bool kNeighbours, int kRows>
__global__ void __launch_bounds__(kThreads) diffrotary_kernel(const __grid_constant__ RotaryParams p) {
  constexpr int kQuads = sizeof(T) / 2;  // 16-byte loads of eight channels
  const uint64_t id = static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const uint64_t token64 = id >> p.unit_bits;
  const int u = static_cast<int>(id & ((1u << p.unit_bits) - 1));
  int slice = blockIdx.y, k = 0;
  while (slice >= p.t[k].slices) slice -= p.t[k++].slices;
  const RotaryTensor &t = p.t[k];
  grid_dependency_wait();
  grid_dependents_launch();
  if (token64 >= p.tokens) return;
  const uint32_t token = static_cast<uint32_t>(token64);
  const uint32_t b = token / p.N, i = token - b * p.N;
  const bool turns = 16 * u < p.rot;
  if (!turns && t.x == t.y) return;  // in place: the other channels stay
  const UnitAt at = unit_at(u, p.rot, kNeighbours);
  const int h0 = slice * kRows;
  const uint8_t *x = t.x + b * t.xb + i * t.xn + h0 * t.xh;
  uint8_t *y = t.y + b * t.yb + i * t.yn + h0 * t.yh;
  uint4 raw[kRows][2 * kQuads];
#pragma unroll
  for (int r = 0; r < kRows; ++r)
    if (h0 + r < t.heads) {
#pragma unroll
      for (int q = 0; q < kQuads; ++q) {
        raw[r][q] = reinterpret_cast<const uint4 *>(x + r * t.xh + at.a * sizeof(T))[q];
        raw[r][kQuads + q] = reinterpret_cast<const uint4 *>(x + r * t.xh + at.b * sizeof(T))[q];
      }
    }
  Turn turn;
  if (turns) {
    int64_t pos = p.positions ? p.positions[b * p.position_stride + i] : p.start + i;
    turn = make_turn<kQuads == 1>(p.freq, u, p.inverse ? -pos : pos, p.scale);
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r)
    if (h0 + r < t.heads) {
      if (turns) {
        float v[16];
        if constexpr (kQuads == 1) {
          widen(raw[r][0], v);
          widen(raw[r][1], v + 8);
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            v[4 * q] = __uint_as_float(raw[r][q].x);
            v[4 * q + 1] = __uint_as_float(raw[r][q].y);
            v[4 * q + 2] = __uint_as_float(raw[r][q].z);
            v[4 * q + 3] = __uint_as_float(raw[r][q].w);
          }
        }
        turn_unit(v, turn, kNeighbours);
        if constexpr (kQuads == 1) {
          raw[r][0] = narrow_bf16(v);
          raw[r][1] = narrow_bf16(v + 8);
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            raw[r][q] = make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]),
                                   __float_as_uint(v[4 * q + 2]), __float_as_uint(v[4 * q + 3]));
        }
      }
      if (!dbg_ok(at.a >= 0 && at.b + 8 <= (16 << p.unit_bits), p.status, 90)) continue;
#pragma unroll
      for (int q = 0; q < kQuads; ++q) {
        reinterpret_cast<uint4 *>(y + r * t.yh + at.a * sizeof(T))[q] = raw[r][q];
        reinterpret_cast<uint4 *>(y + r * t.yh + at.b * sizeof(T))[q] = raw[r][kQuads + q];
      }
    }
}

template <typename T, bool kNeighbours, int kRows>
cudaError_t launch(RotaryParams &p, int count, cudaStream_t stream) {
  unsigned rows = 0;
  for (int k = 0; k < count; ++k) {
    p.t[k].slices = (p.t[k].heads + kRows - 1) / kRows;
    rows += p.t[k].slices;
  }
  const uint64_t threads = static_cast<uint64_t>(p.tokens) << p.unit_bits;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((threads + kThreads - 1) / kThreads), rows);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, diffrotary_kernel<T, kNeighbours, kRows>, p);
}

template <typename T, bool kNeighbours>
cudaError_t launch_rows(RotaryParams &p, int count, int64_t heads, cudaStream_t stream) {
  // Four heads a thread once that still makes two rounds of blocks for every SM; below it the
  // loads of single heads are spread over more SMs.
  const double blocks = std::ldexp(static_cast<double>(p.tokens), p.unit_bits) *
                        static_cast<double>(heads) / (4.0 * kThreads);
  return blocks >= 2 * 152 * 4 ? launch<T, kNeighbours, 4>(p, count, stream)
                               : launch<T, kNeighbours, 1>(p, count, stream);
}

}  // namespace
}  // namespace diffattn

using namespace diffattn;

extern "C" {

diffattn_status diffrotary_frequencies(int32_t rot, double base, int32_t scaling, double factor,
                                       double original, double fast, double slow, uint64_t *freq,
                                       float *scale) {
  if (freq == nullptr || scale == nullptr || rot < 16 || rot % 16 != 0 || !(base > 1.0) ||
      !std::isfinite(base) || scaling < DIFFROTARY_NONE || scaling > DIFFROTARY_PARTS)
    return DIFFATTN_ERR_INVALID_ARG;
  if (scaling != DIFFROTARY_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
    return DIFFATTN_ERR_INVALID_ARG;
  if (scaling == DIFFROTARY_PARTS &&
      (!(original > 0.0) || !std::isfinite(original) || !(slow >= 0.0) || !(fast > slow) ||
       !std::isfinite(fast)))
    return DIFFATTN_ERR_INVALID_ARG;
  const double turn = 2.0 * std::acos(-1.0);
  if (scaling == DIFFROTARY_NTK) base *= std::pow(factor, rot / (rot - 2.0));
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (scaling == DIFFROTARY_LINEAR) f /= factor;
    if (scaling == DIFFROTARY_PARTS) {
      double keep = (original * f / turn - slow) / (fast - slow);
      keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
      f *= keep + (1.0 - keep) / factor;
    }
    freq[i] = static_cast<uint64_t>(std::ldexp(f / turn, 64));  // f <= 1 radian: below 2^62
  }
  *scale = scaling == DIFFROTARY_PARTS ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  return DIFFATTN_OK;
}

diffattn_status diffrotary_apply(const diffattn_desc *desc, const diffrotary_table *table,
                                 int32_t count, const void *const *x, void *const *y,
                                 const int64_t *heads, const diffattn_strides *strides,
                                 const int32_t *positions, int64_t position_stride, int64_t start,
                                 int32_t inverse, void *stream) {
  diffattn_status st = check_common_desc(desc);
  if (st != DIFFATTN_OK) return st;
  if (table == nullptr || count < 1 || count > 4 || x == nullptr || y == nullptr ||
      heads == nullptr || position_stride < 0 || (reinterpret_cast<uintptr_t>(positions) & 3) != 0)
    return DIFFATTN_ERR_INVALID_ARG;
  if (desc->dtype != DIFFATTN_BF16 && desc->dtype != DIFFATTN_F32) return DIFFATTN_ERR_UNSUPPORTED;
  if (desc->d != 64 && desc->d != 128) return DIFFATTN_ERR_UNSUPPORTED;
  if (!rotary_table_ok(*table, desc->d)) return DIFFATTN_ERR_INVALID_ARG;
  const int64_t size = desc->dtype == DIFFATTN_F32 ? 4 : 2, d = desc->d, N = desc->N;
  const double all = static_cast<double>(desc->B) * static_cast<double>(N);
  RotaryParams p = {};
  int used = 0;
  int64_t rows = 0;
  for (int k = 0; k < count; ++k) {
    if (heads[k] < 0 || heads[k] > 65535) return DIFFATTN_ERR_INVALID_ARG;
    if (heads[k] == 0 || all == 0) continue;
    const diffattn_strides xs = strides ? strides[2 * k] : diffattn_strides{heads[k] * N * d, N * d, d};
    const diffattn_strides ys = strides ? strides[2 * k + 1] : xs;
    if (x[k] == nullptr || y[k] == nullptr ||
        ((reinterpret_cast<uintptr_t>(x[k]) | reinterpret_cast<uintptr_t>(y[k])) & 15) != 0 ||
        !paged_strides_ok(xs, 16 / size) || !paged_strides_ok(ys, 16 / size))
      return DIFFATTN_ERR_INVALID_ARG;
    if (x[k] == y[k] && (xs.b != ys.b || xs.h != ys.h || xs.n != ys.n))
      return DIFFATTN_ERR_INVALID_ARG;
    rows += heads[k];
    p.t[used++] = {static_cast<const uint8_t *>(x[k]), static_cast<uint8_t *>(y[k]),
                   xs.b * size, xs.h * size, xs.n * size, ys.b * size, ys.h * size, ys.n * size,
                   static_cast<int32_t>(heads[k]), 0};
  }
  if (used == 0) return DIFFATTN_OK;
  if (all >= 2147483648.0 || rows > 65535) return DIFFATTN_ERR_UNSUPPORTED;
  if ((st = require_sm103()) != DIFFATTN_OK) return st;
  p.freq = table->freq;
  p.positions = positions;
  p.position_stride = position_stride;
  p.start = start;
  p.tokens = static_cast<uint32_t>(desc->B * N);
  p.N = static_cast<uint32_t>(N);
  p.unit_bits = desc->d == 64 ? 2 : 3;
  p.rot = table->rot;
  p.inverse = inverse != 0;
  p.scale = table->scale;
  p.status = desc->status_dev;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (desc->dtype == DIFFATTN_F32)
    e = table->neighbours ? launch_rows<float, true>(p, used, rows, s)
                          : launch_rows<float, false>(p, used, rows, s);
  else
    e = table->neighbours ? launch_rows<__nv_bfloat16, true>(p, used, rows, s)
                          : launch_rows<__nv_bfloat16, false>(p, used, rows, s);
  return e == cudaSuccess ? DIFFATTN_OK : DIFFATTN_ERR_CUDA;
}

}  // extern "C"
