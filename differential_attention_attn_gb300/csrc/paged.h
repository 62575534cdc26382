// Launchers of the paged key/value-cache operators (include/diffattn_paged.h).
// Each takes validated arguments and enqueues its kernels on `stream`.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/diffattn_paged.h"
#include "internal.h"

namespace diffattn {

// Checks shared by the C-ABI files over paged caches (paged_api.cu): strides (positive multiples
// below 2^39), and everything that the desc and the cache say on their own.  query_heads: H
// counts query heads, a multiple of kv_heads, else H = kv_heads.
bool paged_strides_ok(const diffattn_strides &s, int64_t multiple);
diffattn_status check_paged_cache(const diffattn_desc *desc, const diffpaged_cache *c,
                                  bool query_heads);

constexpr int kPageGrain = 16;  // page sizes are multiples of this many rows

// Forward: keys are taken in tiles of kPagedTile; the rows (new token, query
// head) of one key/value head in blocks of 1, 2, 4 .. 32.
constexpr int kPagedTile = 128;
constexpr int kPagedMaxTokens = 16;
constexpr int kPagedMaxGroup = 64;

// How items (sequence, key/value head, row block) go to CTAs: one each; in equal shares of all
// tiles, each item whole in the share that it begins in; in equal shares that cut items, which the
// second kernel joins; or one of these, as the lengths found on the device have it.
enum PagedMode : int32_t { kPagedWhole, kPagedUncut, kPagedCut, kPagedByLengths };

struct PagedFwdPlan {
  int ctas;        // CTAs of the main kernel
  PagedMode mode;  // not kPagedCut: no capacity says that the lengths are long
  int row_tile;    // rows of a block
  int row_blocks;  // row blocks per key/value head
  int64_t items;   // B * kv_heads * row_blocks
  int64_t padded;  // keys per sequence in the logit buffer, a multiple of kPagedTile
  size_t part, stats, item_stats, logits;  // workspace offsets, bytes
  size_t bytes;
};

// False when a size does not fit.
bool plan_paged_fwd(const diffattn_desc &desc, const diffpaged_cache &cache, bool accumulate,
                    int sm_count, PagedFwdPlan *plan);

diffattn_status launch_paged_fwd(const diffattn_desc &desc, const diffpaged_cache &cache,
                                 const PagedFwdPlan &plan, const void *q1, const void *q2,
                                 const float *lambda, const float *norm_w, void *out,
                                 const diffattn_strides *strides, bool accumulate,
                                 void *workspace, cudaStream_t stream);

diffattn_status launch_paged_append(const diffattn_desc &desc, const diffpaged_cache &cache,
                                    const void *k1, const void *k2, const void *v,
                                    const diffattn_strides *strides, cudaStream_t stream);

// False when a size does not fit.
bool paged_evict_bytes(const diffattn_desc &desc, const diffpaged_cache &cache, int64_t keep,
                       size_t *bytes);
diffattn_status launch_paged_evict(const diffattn_desc &desc, const diffpaged_cache &cache,
                                   int64_t keep, int64_t recent, void *workspace,
                                   cudaStream_t stream);

// Exact division of 0 <= n < 2^31 by a launch constant: a multiply and a shift.
struct FastDiv {
  uint32_t mul, shift, d;
  __device__ __forceinline__ int32_t div(int32_t n) const {
    return static_cast<int32_t>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * mul) >> shift);
  }
  __device__ __forceinline__ int32_t mod(int32_t n) const {
    return n - div(n) * static_cast<int32_t>(d);
  }
};
inline FastDiv fast_div(uint32_t d) {  // 2^(s - 1) < d <= 2^s, mul = ceil(2^(31 + s) / d)
  uint32_t s = 0;
  while ((uint64_t{1} << s) < d) ++s;
  return {static_cast<uint32_t>(((uint64_t{1} << (31 + s)) + d - 1) / d), 31 + s, d};
}

// kv_len is read by plain loads and only behind the dependency wait of a kernel or of the one before
// it: diffpaged_evict writes it, and the kernels behind may be resident by then (dependent launch),
// where the read-only path (__ldg) must not be used.

// Stores DIFFATTN_ERR_PAGE in the call's status word unless another code is there.
__device__ __forceinline__ void report_bad_page(int32_t *status) {
  if (status != nullptr) atomicCAS(status, 0, static_cast<int32_t>(DIFFATTN_ERR_PAGE));
}

}  // namespace diffattn
