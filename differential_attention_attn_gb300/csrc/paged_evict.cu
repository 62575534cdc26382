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
//      then writes the list of kept places and moves the weights.  Up to
//      16384 weights are held in shared memory, more in the workspace.
//   2. Move (one block per item and column slice of k1, k2, v).  A
//      kept row's place is at or before its source, and sources ascend, so
//      blocks of rows taken in order only need all loads of a block before
//      its stores; the slices are independent of one another.  The next
//      rows' places are fetched while a block of rows is on its way.
//
// Bound: HBM, each kept row behind the first one dropped read and written once.  16 x 8 heads of 8000 to 8192
// keys at d = 64 cut to 4096 (543 MB): 103 us, the selection 14 us of it and the
// move 86 us, 93 % of the copy rate; 4 x 16 heads of e4m3 keys cut from 1088 to
// 1024: 16 to 17 us, 5.5 us the selection.
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "debug_check.cuh"
#include "paged.h"
#include "ptx.cuh"

namespace diffattn {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048 / kSelectThreads;  // of a histogram, per thread
// 256 rows of a slice a block, two blocks in flight: 103 us for 16 x 8 heads of 8192 keys halved;
// with 256 threads (128 rows, three in flight) 110 us, with slices of 64 bytes 109 us, of 256 bytes
// 129 us.
constexpr int kMoveThreads = 1024;
constexpr int kBatch = 2;   // 16-byte units of a thread in a block of rows
constexpr int kAhead = 2;   // blocks of rows in flight
constexpr size_t kRingBytes = size_t{16} * kAhead * kBatch * kMoveThreads;
constexpr int kHeld = 16384;  // weights that the selection holds in shared memory
constexpr int kMostSlices = 8;  // 128-byte columns of k1, k2 and v rows: 8 d bytes, d <= 128

struct EvictParams {
  uint8_t *pool[3];
  int64_t page_b[3], head_b[3], row_b[3];  // strides in bytes
  int32_t width_b[3];                      // bytes of a row
  int32_t slice_b;                         // of them a block of the move takes
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
  uint32_t x = __float_as_uint(w);
  if ((x & 0x7FFFFFFFu) > 0x7F800000u) x = 0x7F800000u;
  if (x == 0x80000000u) x = 0;
  return x ^ (static_cast<uint32_t>(static_cast<int32_t>(x) >> 31) | 0x80000000u);
}

// Exclusive prefix sum over the block; *total gets the whole sum.  Two barriers; the caller has one
// more between calls that use the same scratch.
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
  // Every warp sums the warps before it.
  const uint32_t mine = lane < kSelectWarps ? scratch[lane] : 0;
  *total = __reduce_add_sync(0xffffffffu, mine);
  return __reduce_add_sync(0xffffffffu, lane < warp ? mine : 0) + incl - x;
}

// The loops are kept rolled: a block runs each once or a few times, so the code that it has to
// fetch counts for more than what it executes (unrolled over weights in registers the same steps
// took 19 us for 128 items of 8192 keys, rolled 14 us).
__global__ void __launch_bounds__(kSelectThreads) diffpaged_select_kernel(const EvictParams p) {
  extern __shared__ float held[];
  __shared__ uint32_t hist[2048];
  __shared__ uint32_t scratch[2][kSelectWarps];
  __shared__ uint32_t found[2];
  const int item = blockIdx.x, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int b = item / p.kv_heads, hk = item % p.kv_heads;
  for (int i = tid; i < 2048; i += kSelectThreads) hist[i] = 0;
  grid_dependency_wait();
  grid_dependents_launch();
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
  const int32_t old = len - p.recent;
  const uint32_t k_keep = p.keep - p.recent;
  float *w = len <= kHeld ? held : p.copy + item * p.padded;  // the weights by position
  const auto weights_of = [&](int32_t page) {
    return p.weights + (static_cast<int64_t>(page) * p.kv_heads + hk) * p.page_size;
  };
  __syncthreads();

  // The k-th largest key, from its leading bits down.
  uint32_t prefix = 0, need = k_keep;  // need: how many are still to be found at or below prefix
  bool bad = false;
  const auto count = [&](float x, int32_t j, int shift, int bits) {
    const uint32_t key = order_key(x);
    if (j < old && (shift + bits >= 32 || (key ^ prefix) >> (shift + bits) == 0))
      atomicAdd(&hist[(key >> shift) & ((1u << bits) - 1)], 1u);
  };
#pragma unroll 4
  for (int32_t j = tid; j < len; j += kSelectThreads) {
    const int32_t n = p.by_page.div(j);
    const int32_t page = __ldg(table + n);
    if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.num_pages)) {
      bad = true;
    } else {
      const float x = weights_of(page)[j - n * p.page_size];
      w[j] = x;
      count(x, j, 21, 11);
    }
  }
  if (__syncthreads_or(bad)) {  // a page of the sequence is not one: it stays as it is
    if (tid == 0) {
      report_bad_page(p.status);
      p.plan[item] = make_int2(0, 0);
    }
    return;
  }
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass < 2 ? 11 : 10;
    if (pass > 0) {
#pragma unroll 1
      for (int32_t j = tid; j < old; j += kSelectThreads) count(w[j], j, shift, bits);
      __syncthreads();
    }
    // Thread t holds the kBins bins below 2048 - kBins t: sums from the largest bin down.
    uint32_t bin_of[kBins], mine = 0;
#pragma unroll
    for (int k = 0; k < kBins; ++k) {
      bin_of[k] = hist[2047 - kBins * tid - k];
      hist[2047 - kBins * tid - k] = 0;
      mine += bin_of[k];
    }
    if (tid == 0) found[0] = found[1] = 0;
    uint32_t total;
    uint32_t above = block_scan(mine, scratch[0], &total);
#pragma unroll
    for (int k = 0; k < kBins; ++k) {
      if (need > above && need <= above + bin_of[k]) {
        found[0] = 2047 - kBins * tid - k;
        found[1] = need - above;
      }
      above += bin_of[k];
    }
    __syncthreads();
    prefix |= found[0] << shift;
    need = found[1];
  }
  if (k_keep == 0) prefix = 0xFFFFFFFFu;  // above every key

  // Kept places in order: keys above T, the first `need` equal to it, and the last `recent`.  Each
  // warp has a run of positions, 32 a step; the warps before it tell it where its own go.
  const int32_t steps = (len + 32 * kSelectWarps - 1) / (32 * kSelectWarps);
  const int32_t from = warp * steps * 32, to = min(len, from + steps * 32);
  uint32_t above_t = 0, equal_t = 0;
#pragma unroll 1
  for (int32_t j0 = from; j0 < to; j0 += 32) {
    const int32_t j = j0 + lane;
    const uint32_t key = j < old ? order_key(w[j]) : 0;
    above_t += __popc(__ballot_sync(0xffffffffu, j < to && (j >= old || key > prefix)));
    equal_t += __popc(__ballot_sync(0xffffffffu, j < old && j < to && key == prefix));
  }
  if (lane == 0) {
    scratch[0][warp] = above_t;
    scratch[1][warp] = equal_t;
  }
  __syncthreads();
  const bool before = lane < warp && lane < kSelectWarps;
  uint32_t equal_before = __reduce_add_sync(0xffffffffu, before ? scratch[1][lane] : 0);
  uint32_t at = __reduce_add_sync(0xffffffffu, before ? scratch[0][lane] : 0) +
                min(need, equal_before);
  int2 *list = p.list + static_cast<int64_t>(item) * p.keep;
  const uint32_t lower = (1u << lane) - 1;
  uint32_t in_place = 0xFFFFFFFFu;  // the first position that does not stay
#pragma unroll 1
  for (int32_t j0 = from; j0 < to; j0 += 32) {
    const int32_t j = j0 + lane;
    const float x = j < to ? w[j] : 0.f;
    const uint32_t key = j < old ? order_key(x) : 0;
    const bool is_equal = j < old && j < to && key == prefix;
    const uint32_t equals = __ballot_sync(0xffffffffu, is_equal);
    const bool stays =
        j < to && (j >= old || key > prefix ||
                   (is_equal && equal_before + __popc(equals & lower) < need));
    const uint32_t kept = __ballot_sync(0xffffffffu, stays);
    const uint32_t dst = at + __popc(kept & lower);
    if (stays && dbg_ok(dst < static_cast<uint32_t>(p.keep), p.status, 50)) {
      const int32_t n = p.by_page.div(j), m = p.by_page.div(static_cast<int32_t>(dst));
      list[dst] = make_int2(__ldg(table + n), j - n * p.page_size);
      weights_of(__ldg(table + m))[static_cast<int32_t>(dst) - m * p.page_size] = x;
    }
    const uint32_t gone = __ballot_sync(0xffffffffu, j < to && !stays);
    if (gone) in_place = min(in_place, static_cast<uint32_t>(j0 + __ffs(gone) - 1));
    equal_before += __popc(equals);
    at += __popc(kept);
  }
  __syncthreads();
  if (lane == 0) scratch[0][warp] = in_place;
  __syncthreads();
  if (warp == 0) {
    in_place = __reduce_min_sync(0xffffffffu, lane < kSelectWarps ? scratch[0][lane] : 0xFFFFFFFFu);
    if (lane == 0) p.plan[item] = make_int2(min(static_cast<int32_t>(in_place), p.keep), 1);
  }
}

__host__ __device__ __forceinline__ int32_t slices_of(int32_t width, int32_t slice) {
  return (width + slice - 1) / slice;
}

__global__ void __launch_bounds__(kMoveThreads) diffpaged_move_kernel(const EvictParams p,
                                                                      int slices) {
  const int item = blockIdx.x / slices;
  int slice = blockIdx.x - item * slices;
  const int b = item / p.kv_heads, hk = item - b * p.kv_heads;
  int t = 0;
  while (slice >= slices_of(p.width_b[t], p.slice_b)) slice -= slices_of(p.width_b[t++], p.slice_b);
  const int units = min(p.width_b[t], p.slice_b) / 16;  // 16-byte units of the slice
  const int unit = threadIdx.x & (units - 1), line = threadIdx.x / units;
  const int lines = kMoveThreads / units;  // rows taken side by side
  uint8_t *base = p.pool[t] + hk * p.head_b[t] + slice * p.slice_b + unit * 16;
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
  extern __shared__ uint4 ring_raw[];
  auto *ring = reinterpret_cast<uint4(*)[kBatch][kMoveThreads]>(ring_raw);
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

// For a budget that no sequence can pass: the lengths are looked at all the same.
__global__ void __launch_bounds__(256)
    diffpaged_lengths_kernel(const int32_t *kv_len, int32_t B, int32_t most, int32_t *status) {
  grid_dependency_wait();
  const uint32_t b = blockIdx.x * 256 + threadIdx.x;
  if (b < static_cast<uint32_t>(B) && (kv_len[b] < 0 || kv_len[b] > most)) report_bad_page(status);
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
  const int64_t copied = most > kHeld ? most : 0;
  l.list = round256(static_cast<size_t>(items * copied) * sizeof(float));
  l.plan = l.list + round256(static_cast<size_t>(items * kept) * sizeof(int2));
  l.bytes = l.plan + round256(static_cast<size_t>(items) * sizeof(int2));
  return l;
}

}  // namespace

bool paged_evict_bytes(const diffattn_desc &desc, const diffpaged_cache &cache, int64_t keep,
                       size_t *bytes) {
  *bytes = 0;
  const int64_t most = cache.max_pages * cache.page_size;
  // A budget that no sequence can pass needs nothing.
  if (keep >= most || desc.B == 0) return true;
  const double items = static_cast<double>(desc.B) * static_cast<double>(cache.kv_heads);
  if (items * kMostSlices > INT32_MAX || items * static_cast<double>(most) > 1.0e17) return false;
  *bytes = layout(desc, cache, keep).bytes;
  return true;
}

diffattn_status launch_paged_evict(const diffattn_desc &desc, const diffpaged_cache &cache,
                                   int64_t keep, int64_t recent, void *workspace,
                                   cudaStream_t stream) {
  const int64_t most = cache.max_pages * cache.page_size;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (keep >= most) {
    if (desc.status_dev == nullptr) return DIFFATTN_OK;
    cfg.gridDim = dim3(static_cast<unsigned>((desc.B + 255) / 256));
    cfg.blockDim = dim3(256);
    return cudaLaunchKernelEx(&cfg, diffpaged_lengths_kernel,
                              static_cast<const int32_t *>(cache.kv_len),
                              static_cast<int32_t>(desc.B), static_cast<int32_t>(most),
                              desc.status_dev) == cudaSuccess
               ? DIFFATTN_OK
               : DIFFATTN_ERR_CUDA;
  }
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
  }
  // Slices of 128 bytes, narrower ones (down to a sector) while some SMs would have none: 8192 keys
  // halved, 8 heads 30.5 -> 23.5 us, 32 heads 46.7 -> 41 us.
  const int sms = device_sm_count();
  if (sms <= 0) return DIFFATTN_ERR_CUDA;
  for (p.slice_b = 128;; p.slice_b /= 2) {
    slices = 0;
    for (int t = 0; t < 3; ++t) slices += slices_of(p.width_b[t], p.slice_b);
    if (p.slice_b == 32 || desc.B * cache.kv_heads * slices > sms) break;
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
  const int64_t items = desc.B * cache.kv_heads;  // items * kMostSlices fits (paged_evict_bytes)
  cfg.gridDim = dim3(static_cast<unsigned>(items));
  cfg.blockDim = dim3(kSelectThreads);
  cfg.dynamicSmemBytes = sizeof(float) * static_cast<size_t>(most < kHeld ? most : kHeld);
  static std::atomic<bool> attr_set[64];  // per device (concurrent callers may both set)
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DIFFATTN_ERR_CUDA;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(diffpaged_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(sizeof(float) * kHeld)) != cudaSuccess ||
        cudaFuncSetAttribute(diffpaged_move_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kRingBytes)) != cudaSuccess)
      return DIFFATTN_ERR_CUDA;
    attr_set[dev].store(true, std::memory_order_release);
  }
  if (cudaLaunchKernelEx(&cfg, diffpaged_select_kernel, p) != cudaSuccess) return DIFFATTN_ERR_CUDA;
  cfg.gridDim = dim3(static_cast<unsigned>(items) * slices);
  cfg.blockDim = dim3(kMoveThreads);
  cfg.dynamicSmemBytes = kRingBytes;
  return cudaLaunchKernelEx(&cfg, diffpaged_move_kernel, p, slices) == cudaSuccess
             ? DIFFATTN_OK
             : DIFFATTN_ERR_CUDA;
}

}  // namespace diffattn
