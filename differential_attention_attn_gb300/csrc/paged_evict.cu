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
//      then writes the list of kept positions and moves the weights.
//   2. Move (one block per item and 128-byte column slice of k1, k2, v).  A
//      kept row's place is at or before its source, and sources ascend, so
//      blocks of rows taken in order only need all loads of a block before
//      its stores; the slices are independent of one another.
//
// Bound: HBM, each kept row read and written once; the selection reads the
// weights once and then works in the cache.
#include <cuda_runtime.h>

#include <cstdint>

#include "debug_check.cuh"
#include "paged.h"
#include "ptx.cuh"

namespace diffattn {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int kBatch = 8;  // 16-byte units a thread has in flight

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
  int64_t padded;   // entries per item of copy
  float *copy;      // [items][padded] the item's weights, by position
  int32_t *list;    // [items][keep] source position of each kept row
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

__global__ void __launch_bounds__(kSelectThreads) diffpaged_select_kernel(const EvictParams p) {
  __shared__ uint32_t hist[2048];
  __shared__ uint32_t scratch[32];
  __shared__ uint32_t found[2];
  grid_dependents_launch();
  const int item = blockIdx.x, tid = threadIdx.x;
  const int b = item / p.kv_heads, hk = item % p.kv_heads;
  const int32_t len = p.kv_len[b];
  const bool bad_len = len < 0 || len > p.max_pages * p.page_size;
  if (bad_len || len <= p.keep) {
    if (tid == 0) {
      if (bad_len) report_bad_page(p.status);
      p.plan[item] = make_int2(0, 0);
    }
    return;
  }
  const int32_t *table = p.page_table + static_cast<int64_t>(b) * p.max_pages;
  bool bad = false;
  for (int k = tid; k * p.page_size < len; k += kSelectThreads)
    bad |= static_cast<uint32_t>(table[k]) >= static_cast<uint32_t>(p.num_pages);
  if (__syncthreads_or(bad)) {
    if (tid == 0) {
      report_bad_page(p.status);
      p.plan[item] = make_int2(0, 0);
    }
    return;
  }
  const int32_t old = len - p.recent;
  const uint32_t k_keep = p.keep - p.recent;
  float *copy = p.copy + item * p.padded;
  const auto weight_at = [&](int32_t j) -> float * {
    return p.weights + (static_cast<int64_t>(table[j / p.page_size]) * p.kv_heads + hk) * p.page_size +
           j % p.page_size;
  };

  // The k-th largest key, from its leading bits down.
  uint32_t prefix = 0, need = k_keep;  // need: how many are still to be found at or below prefix
  const int shift[3] = {21, 10, 0}, bits[3] = {11, 11, 10};
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    for (int i = tid; i < 2048; i += kSelectThreads) hist[i] = 0;
    __syncthreads();
    const uint32_t high = pass == 0 ? 0 : prefix >> (shift[pass] + bits[pass]);
    for (int32_t j = tid; j < (pass == 0 ? len : old); j += kSelectThreads) {
      float w;
      if (pass == 0)
        copy[j] = w = *weight_at(j);
      else
        w = copy[j];
      const uint32_t key = order_key(w);
      if (j < old && (pass == 0 || key >> (shift[pass] + bits[pass]) == high))
        atomicAdd(&hist[(key >> shift[pass]) & ((1u << bits[pass]) - 1)], 1u);
    }
    __syncthreads();
    // Thread t holds bins 2047 - 2 t and 2046 - 2 t: sums from the largest bin down.
    const uint32_t hi = hist[2047 - 2 * tid], lo = hist[2046 - 2 * tid];
    uint32_t total;
    const uint32_t above = block_scan(hi + lo, scratch, &total);
    if (tid == 0) found[0] = found[1] = 0;
    __syncthreads();
    if (need > above && need <= above + hi + lo) {
      const bool in_hi = need <= above + hi;
      found[0] = in_hi ? 2047 - 2 * tid : 2046 - 2 * tid;
      found[1] = need - above - (in_hi ? 0 : hi);
    }
    __syncthreads();
    prefix |= found[0] << shift[pass];
    need = found[1];
    __syncthreads();
  }

  // Kept positions in order: keys above T, and the first `need` equal to it.
  uint32_t equal_before = 0, kept = 0;
  int32_t *list = p.list + static_cast<int64_t>(item) * p.keep;
  uint32_t in_place = 0;  // leading positions that all stay
  for (int32_t j0 = 0; j0 < old; j0 += kSelectThreads) {
    const int32_t j = j0 + tid;
    const float w = j < old ? copy[j] : 0.f;
    const uint32_t key = j < old ? order_key(w) : 0;
    const bool equal = k_keep > 0 && j < old && key == prefix;
    uint32_t total, all_equal;
    const uint32_t eq = block_scan(equal, scratch, &all_equal);
    const bool stays = k_keep > 0 && j < old && (key > prefix || (equal && equal_before + eq < need));
    const uint32_t at = kept + block_scan(stays, scratch, &total);
    if (stays && dbg_ok(at < k_keep, p.status, 50)) {
      list[at] = j;
      *weight_at(static_cast<int32_t>(at)) = w;
    }
    if (in_place == static_cast<uint32_t>(j0) && total == static_cast<uint32_t>(kSelectThreads))
      in_place = j0 + kSelectThreads;
    equal_before += all_equal;
    kept += total;
  }
  for (int32_t j = old + tid; j < len; j += kSelectThreads) {
    const int32_t at = static_cast<int32_t>(k_keep) + j - old;
    list[at] = j;
    *weight_at(at) = copy[j];
  }
  if (tid == 0) p.plan[item] = make_int2(static_cast<int32_t>(in_place), 1);
}

__global__ void __launch_bounds__(kMoveThreads) diffpaged_move_kernel(const EvictParams p,
                                                                      int slices) {
  grid_dependency_wait();
  const int item = blockIdx.x / slices;
  int slice = blockIdx.x % slices;
  const int b = item / p.kv_heads, hk = item % p.kv_heads;
  const int2 plan = p.plan[item];
  if (plan.y == 0) return;
  if (slice == 0 && hk == 0 && threadIdx.x == 0) p.kv_len[b] = p.keep;
  int t = 0;
  while (slice >= (p.width_b[t] + 127) / 128) slice -= (p.width_b[t++] + 127) / 128;
  const int units = p.width_b[t] < 128 ? p.width_b[t] / 16 : 8;  // 16-byte units of the slice
  const int unit = threadIdx.x % units, line = threadIdx.x / units;
  const int lines = kMoveThreads / units;  // rows taken side by side
  uint8_t *base = p.pool[t] + hk * p.head_b[t] + slice * 128 + unit * 16;
  const int32_t *table = p.page_table + static_cast<int64_t>(b) * p.max_pages;
  const int32_t *list = p.list + static_cast<int64_t>(item) * p.keep;
  const auto row_at = [&](int32_t j) {
    return reinterpret_cast<uint4 *>(base + table[j / p.page_size] * p.page_b[t] +
                                     j % p.page_size * p.row_b[t]);
  };
  for (int32_t first = plan.x; first < p.keep; first += lines * kBatch) {
    uint4 x[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int32_t at = first + u * lines + line;
      if (at < p.keep) x[u] = *row_at(list[at]);
    }
    __syncthreads();  // every source of these rows is read before any of their places is written
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int32_t at = first + u * lines + line;
      if (at < p.keep) *row_at(at) = x[u];
    }
  }
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
  l.list = round256(static_cast<size_t>(items * most) * sizeof(float));
  l.plan = l.list + round256(static_cast<size_t>(items * kept) * sizeof(int32_t));
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
  p.padded = l.padded;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  p.copy = reinterpret_cast<float *>(ws + l.copy);
  p.list = reinterpret_cast<int32_t *>(ws + l.list);
  p.plan = reinterpret_cast<int2 *>(ws + l.plan);
  const double items = static_cast<double>(desc.B) * static_cast<double>(cache.kv_heads);
  if (items * slices > INT32_MAX) return DIFFATTN_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items));
  cfg.blockDim = dim3(kSelectThreads);
  cfg.stream = stream;
  if (cudaLaunchKernelEx(&cfg, diffpaged_select_kernel, p) != cudaSuccess) return DIFFATTN_ERR_CUDA;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(items) * slices);
  cfg.blockDim = dim3(kMoveThreads);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, diffpaged_move_kernel, p, slices) == cudaSuccess
             ? DIFFATTN_OK
             : DIFFATTN_ERR_CUDA;
}

}  // namespace diffattn
