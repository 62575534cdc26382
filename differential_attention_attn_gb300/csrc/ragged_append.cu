// diffragged_append: the packed tokens' queries turned, their keys turned and
// written to the cache with the values.
//
// Token t goes to row slot % page_size of page slot / page_size.  Queries and
// keys are widened, turned by the token's position and rounded once (bf16, or
// e4m3 saturating at +-448); values are copied.
//
// Bound: a read and a write of every row, so HBM bandwidth for prompts and the
// chain slot -> store for single tokens.  A thread has one unit (16 channels) of
// one token in kRows heads of one tensor (a value row counts as two heads), so
// that the sines are worked out once for all of them and their loads are on
// their way together (two heads 36.9 us, four 34.8, eight 40.9 for 221 MB), in
// small blocks at full occupancy (256 threads at three blocks an SM: 38.0 us).
// Measured on GB300: 9004 tokens of 32 heads over 8 key/value heads at d = 64,
// 221 MB: 34.8 us, 94 % of the copy rate; 6165 tokens at d = 128 with e4m3 keys,
// 120 MB: 23.8 us, 74 %; 64 single tokens 2.1 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "debug_check.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "ragged.h"
#include "rotary.cuh"

namespace diffattn {
namespace {

constexpr int kThreads = 128;
enum : int { kQ1, kQ2, kK1, kK2, kV, kTensors };

struct RaggedAppendParams {
  const uint8_t *src[kTensors];
  uint8_t *dst[kTensors];  // the outputs of q1, q2, the pools of k1, k2, v
  int64_t src_n[kTensors], src_h[kTensors];  // byte strides
  int64_t dst_n[kTensors], dst_h[kTensors], dst_p[kTensors];  // dst_p: of a page
  int32_t heads[kTensors], slices[kTensors];  // rows of a token; slices of kRows of them
  const int64_t *slots;
  const int32_t *positions;
  const uint64_t *freq;
  float *weights;
  int32_t *status;
  uint32_t tokens;
  int32_t rot, kv_heads, page_size;  // rot 0: nothing is turned
  int64_t places;                    // num_pages * page_size
  FastDiv by_page, by_slices;
  float scale;
};

template <int kD, bool kFp8, bool kNeighbours, int kRows>
__global__ void __launch_bounds__(kThreads, 8)
    diffragged_append_kernel(const __grid_constant__ RaggedAppendParams p) {
  constexpr int kUnits = kD / 16;
  // The slices of the same tokens in neighbouring blocks: their rows lie side by side.
  const uint32_t tokens = p.by_slices.div(blockIdx.x);
  const uint32_t token = tokens * (kThreads / kUnits) + threadIdx.x / kUnits;
  const int u = threadIdx.x % kUnits;
  int slice = blockIdx.x - tokens * p.by_slices.d, k = 0;
  while (slice >= p.slices[k]) slice -= p.slices[k++];
  grid_dependency_wait();
  grid_dependents_launch();
  if (token >= p.tokens) return;
  const int64_t slot = p.slots[token];
  const int h0 = slice * kRows, heads = p.heads[k];
  const bool is_v = k == kV, turns = !is_v && 16 * u < p.rot;
  const UnitAt at = unit_at(u, is_v ? 0 : p.rot, kNeighbours);
  const uint8_t *x = p.src[k] + token * p.src_n[k];
  uint4 raw[kRows][2];
  // A value row is two rows of kD channels.
  const auto head_at = [&](int64_t stride, int h, int bytes) {
    return is_v ? (h >> 1) * stride + (h & 1) * (kD * bytes) : h * stride;
  };
#pragma unroll
  for (int r = 0; r < kRows; ++r)
    if (h0 + r < heads) {
      const uint8_t *row = x + head_at(p.src_h[k], h0 + r, 2);
      raw[r][0] = *reinterpret_cast<const uint4 *>(row + at.a * 2);
      raw[r][1] = *reinterpret_cast<const uint4 *>(row + at.b * 2);
    }
  if (slot < 0 || slot >= p.places) {
    if (slot != -1) report_bad_page(p.status);
    return;
  }
  Turn turn;
  if (turns) turn = make_turn<!kFp8>(p.freq, u, p.positions[token], p.scale);
  int64_t page = 0;
  int32_t place = 0;
  uint8_t *y = p.dst[k];
  if (k >= kK1) {
    page = slot < (int64_t{1} << 31) ? p.by_page.div(static_cast<int32_t>(slot))
                                     : slot / p.page_size;
    place = static_cast<int32_t>(slot - page * p.page_size);
    y += page * p.dst_p[k] + place * p.dst_n[k];
  } else {
    y += token * p.dst_n[k];
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r)
    if (h0 + r < heads) {
      const int h = h0 + r;
      if (kFp8 && !is_v) {
        float v[16];
        widen(raw[r][0], v);
        widen(raw[r][1], v + 8);
        if (turns) turn_unit(v, turn, kNeighbours);
        uint8_t *row = y + head_at(p.dst_h[k], h, 1);
        *reinterpret_cast<uint2 *>(row + at.a) = narrow_e4m3(v);
        *reinterpret_cast<uint2 *>(row + at.b) = narrow_e4m3(v + 8);
      } else {
        if (turns) {
          float v[16];
          widen(raw[r][0], v);
          widen(raw[r][1], v + 8);
          turn_unit(v, turn, kNeighbours);
          raw[r][0] = narrow_bf16(v);
          raw[r][1] = narrow_bf16(v + 8);
        }
        uint8_t *row = y + head_at(p.dst_h[k], h, 2);
        *reinterpret_cast<uint4 *>(row + at.a * 2) = raw[r][0];
        *reinterpret_cast<uint4 *>(row + at.b * 2) = raw[r][1];
      }
      if (is_v && p.weights != nullptr && u == 0 && (h & 1) == 0 &&
          dbg_ok(place >= 0 && place < p.page_size, p.status, 92))
        p.weights[(page * p.kv_heads + (h >> 1)) * p.page_size + place] = 0.f;
    }
}

template <int kD, bool kFp8, bool kNeighbours, int kRows>
cudaError_t launch_rows(RaggedAppendParams &p, cudaStream_t stream) {
  unsigned slices = 0;
  for (int k = 0; k < kTensors; ++k) {
    p.slices[k] = (p.heads[k] + kRows - 1) / kRows;
    slices += p.slices[k];
  }
  constexpr uint32_t kTokens = kThreads / (kD / 16);
  cudaLaunchConfig_t cfg = {};
  p.by_slices = fast_div(slices);
  cfg.gridDim = dim3((p.tokens + kTokens - 1) / kTokens * slices);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, diffragged_append_kernel<kD, kFp8, kNeighbours, kRows>, p);
}

// Four heads a thread once that still makes two rounds of blocks for every SM; below it the loads of
// single heads are spread over more SMs.
template <int kD, bool kFp8, bool kNeighbours>
cudaError_t launch(RaggedAppendParams &p, cudaStream_t stream) {
  double rows = 0;
  for (int k = 0; k < kTensors; ++k) rows += p.heads[k];
  const double blocks = rows * p.tokens * (kD / 16) / (4.0 * kThreads);
  return blocks >= 2 * 152 * 8 ? launch_rows<kD, kFp8, kNeighbours, 4>(p, stream)
                               : launch_rows<kD, kFp8, kNeighbours, 1>(p, stream);
}

template <int kD, bool kFp8>
cudaError_t launch(RaggedAppendParams &p, bool neighbours, cudaStream_t stream) {
  return neighbours ? launch<kD, kFp8, true>(p, stream) : launch<kD, kFp8, false>(p, stream);
}

}  // namespace

diffattn_status launch_ragged_append(const diffattn_desc &desc, const diffpaged_cache &cache,
                                     const void *const src[5], void *const q_out[2],
                                     const diffattn_strides strides[7], const int64_t *slots,
                                     const diffrotary_table *table, const int32_t *positions,
                                     cudaStream_t stream) {
  const bool fp8 = desc.dtype == DIFFATTN_E4M3_QK;
  RaggedAppendParams p = {};
  const diffattn_strides *pool[3] = {&cache.k1_strides, &cache.k2_strides, &cache.v_strides};
  void *const dst[5] = {q_out[0], q_out[1], cache.k1, cache.k2, cache.v};
  for (int k = 0; k < kTensors; ++k) {
    const int64_t size = fp8 && k != kV ? 1 : 2;
    p.src[k] = static_cast<const uint8_t *>(src[k]);
    p.dst[k] = static_cast<uint8_t *>(dst[k]);
    p.src_n[k] = 2 * strides[k].n;
    p.src_h[k] = 2 * strides[k].h;
    const diffattn_strides &out = k < kK1 ? strides[5 + k] : *pool[k - kK1];
    p.dst_n[k] = size * out.n;
    p.dst_h[k] = size * out.h;
    p.dst_p[k] = k < kK1 ? 0 : size * out.b;
    p.heads[k] = static_cast<int32_t>(k < kK1 ? (src[k] ? desc.H : 0)
                                              : cache.kv_heads * (k == kV ? 2 : 1));
  }
  p.slots = slots;
  p.positions = positions;
  p.weights = cache.weights;
  p.status = desc.status_dev;
  p.tokens = static_cast<uint32_t>(desc.N);
  p.kv_heads = static_cast<int32_t>(cache.kv_heads);
  p.page_size = cache.page_size;
  p.places = cache.num_pages * cache.page_size;
  p.by_page = fast_div(static_cast<uint32_t>(p.page_size));
  if (table != nullptr) {
    p.rot = table->rot;
    p.freq = table->freq;
    p.scale = table->scale;
  }
  const bool neighbours = table != nullptr && table->neighbours;
  const cudaError_t e =
      desc.d == 64 ? (fp8 ? launch<64, true>(p, neighbours, stream)
                          : launch<64, false>(p, neighbours, stream))
                   : (fp8 ? launch<128, true>(p, neighbours, stream)
                          : launch<128, false>(p, neighbours, stream));
  return e == cudaSuccess ? DIFFATTN_OK : DIFFATTN_ERR_CUDA;
}

}  // namespace diffattn
