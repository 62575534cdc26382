// C ABI of the paged key/value-cache operators: argument validation and
// dispatch.  Every entry point is declared, with its contract, in
// include/diffattn_paged.h.
#include <cuda_runtime.h>

#include <cstdint>

#include "paged.h"

namespace {

using namespace diffattn;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kStrideLimit = int64_t{1} << 39;

bool strides_ok(const diffattn_strides &s, int64_t multiple) {
  for (const int64_t x : {s.b, s.h, s.n})
    if (x <= 0 || x % multiple != 0 || x >= kStrideLimit) return false;
  return true;
}

// Everything that the desc and the cache say on their own.  query_heads: H
// counts query heads, a multiple of kv_heads (fwd), else H = kv_heads.
diffattn_status check_cache(const diffattn_desc *desc, const diffpaged_cache *c, bool query_heads) {
  diffattn_status st = check_common_desc(desc);
  if (st != DIFFATTN_OK) return st;
  if (c == nullptr) return DIFFATTN_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->kv_heads < 1 || c->max_pages < 1 || c->page_size < 1 ||
      c->reserved != 0)
    return DIFFATTN_ERR_INVALID_ARG;
  if (query_heads ? desc->H % c->kv_heads != 0 : desc->H != c->kv_heads)
    return DIFFATTN_ERR_INVALID_ARG;
  if (desc->dtype != DIFFATTN_BF16 && desc->dtype != DIFFATTN_E4M3_QK)
    return DIFFATTN_ERR_UNSUPPORTED;
  if (desc->d != 64 && desc->d != 128) return DIFFATTN_ERR_UNSUPPORTED;
  if (c->page_size % kPageGrain != 0) return DIFFATTN_ERR_UNSUPPORTED;
  if (c->num_pages > INT32_MAX || c->kv_heads > 65535 || desc->B > INT32_MAX ||
      c->max_pages >= (int64_t{1} << 30) / c->page_size)
    return DIFFATTN_ERR_UNSUPPORTED;
  if (desc->B == 0 || desc->H == 0) return DIFFATTN_OK;
  if (!c->k1 || !c->k2 || !c->v || !c->page_table || !c->kv_len) return DIFFATTN_ERR_INVALID_ARG;
  if (!aligned(c->k1, 16) || !aligned(c->k2, 16) || !aligned(c->v, 16) ||
      !aligned(c->weights, 4) || !aligned(c->page_table, 4) || !aligned(c->kv_len, 4))
    return DIFFATTN_ERR_INVALID_ARG;
  const int64_t k_multiple = desc->dtype == DIFFATTN_E4M3_QK ? 16 : 8;
  if (!strides_ok(c->k1_strides, k_multiple) || !strides_ok(c->k2_strides, k_multiple) ||
      !strides_ok(c->v_strides, 8))
    return DIFFATTN_ERR_INVALID_ARG;
  return DIFFATTN_OK;
}

diffattn_status plan_fwd(const diffattn_desc *desc, const diffpaged_cache *cache, int accumulate,
                         PagedFwdPlan *plan) {
  diffattn_status st = check_cache(desc, cache, true);
  if (st != DIFFATTN_OK) return st;
  if (accumulate && cache->weights == nullptr) return DIFFATTN_ERR_INVALID_ARG;
  if (desc->N > kPagedMaxTokens || desc->H / cache->kv_heads > kPagedMaxGroup)
    return DIFFATTN_ERR_UNSUPPORTED;
  *plan = PagedFwdPlan{};
  if (desc->B * desc->H * desc->N == 0) return DIFFATTN_OK;
  const int sms = device_sm_count();
  if (sms <= 0) return DIFFATTN_ERR_CUDA;
  return plan_paged_fwd(*desc, *cache, accumulate != 0, sms, plan) ? DIFFATTN_OK
                                                                    : DIFFATTN_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" {

diffattn_status diffpaged_append(const diffattn_desc *desc, const diffpaged_cache *cache,
                                 const void *k1, const void *k2, const void *v,
                                 const diffattn_strides *strides, void *stream) {
  diffattn_status st = check_cache(desc, cache, false);
  if (st != DIFFATTN_OK) return st;
  if (desc->B * desc->H * desc->N == 0) return DIFFATTN_OK;
  if (!k1 || !k2 || !v || !aligned(k1, 16) || !aligned(k2, 16) || !aligned(v, 16))
    return DIFFATTN_ERR_INVALID_ARG;
  if (strides != nullptr)
    for (int i = 0; i < 3; ++i)
      if (!strides_ok(strides[i], 8)) return DIFFATTN_ERR_INVALID_ARG;
  if (desc->N >= (int64_t{1} << 30)) return DIFFATTN_ERR_UNSUPPORTED;
  if ((st = require_sm103()) != DIFFATTN_OK) return st;
  return launch_paged_append(*desc, *cache, k1, k2, v, strides, static_cast<cudaStream_t>(stream));
}

diffattn_status diffpaged_fwd_plan(const diffattn_desc *desc, const diffpaged_cache *cache,
                                   int accumulate, size_t *workspace_bytes) {
  if (workspace_bytes == nullptr) return DIFFATTN_ERR_INVALID_ARG;
  PagedFwdPlan plan;
  const diffattn_status st = plan_fwd(desc, cache, accumulate, &plan);
  if (st == DIFFATTN_OK) *workspace_bytes = plan.bytes;
  return st;
}

diffattn_status diffpaged_fwd(const diffattn_desc *desc, const diffpaged_cache *cache,
                              const void *q1, const void *q2, const float *lambda,
                              const float *norm_w, void *out, const diffattn_strides *strides,
                              int accumulate, void *workspace, size_t workspace_bytes,
                              void *stream) {
  PagedFwdPlan plan;
  diffattn_status st = plan_fwd(desc, cache, accumulate, &plan);
  if (st != DIFFATTN_OK) return st;
  if (desc->B * desc->H * desc->N == 0) return DIFFATTN_OK;
  if (!q1 || !q2 || !lambda || !out || !aligned(q1, 16) || !aligned(q2, 16) || !aligned(out, 16) ||
      !aligned(lambda, 4) || !aligned(norm_w, 4))
    return DIFFATTN_ERR_INVALID_ARG;
  if (strides != nullptr) {
    const int64_t q_multiple = desc->dtype == DIFFATTN_E4M3_QK ? 16 : 8;
    if (!strides_ok(strides[0], q_multiple) || !strides_ok(strides[1], q_multiple) ||
        !strides_ok(strides[2], 8))
      return DIFFATTN_ERR_INVALID_ARG;
  }
  if (plan.bytes > 0 &&
      (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < plan.bytes))
    return DIFFATTN_ERR_INVALID_ARG;
  if ((st = require_sm103()) != DIFFATTN_OK) return st;
  return launch_paged_fwd(*desc, *cache, plan, q1, q2, lambda, norm_w, out, strides,
                          accumulate != 0, workspace, static_cast<cudaStream_t>(stream));
}

diffattn_status diffpaged_evict_plan(const diffattn_desc *desc, const diffpaged_cache *cache,
                                     int64_t keep, size_t *workspace_bytes) {
  diffattn_status st = check_cache(desc, cache, false);
  if (st != DIFFATTN_OK) return st;
  if (workspace_bytes == nullptr || keep < 0 || cache->weights == nullptr)
    return DIFFATTN_ERR_INVALID_ARG;
  return paged_evict_bytes(*desc, *cache, keep, workspace_bytes) ? DIFFATTN_OK
                                                                 : DIFFATTN_ERR_UNSUPPORTED;
}

diffattn_status diffpaged_evict(const diffattn_desc *desc, const diffpaged_cache *cache,
                                int64_t keep, int64_t recent, void *workspace,
                                size_t workspace_bytes, void *stream) {
  size_t need = 0;
  diffattn_status st = diffpaged_evict_plan(desc, cache, keep, &need);
  if (st != DIFFATTN_OK) return st;
  if (recent < 0 || recent > keep) return DIFFATTN_ERR_INVALID_ARG;
  if (desc->B * desc->H == 0) return DIFFATTN_OK;
  if (need > 0 && (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < need))
    return DIFFATTN_ERR_INVALID_ARG;
  if ((st = require_sm103()) != DIFFATTN_OK) return st;
  return launch_paged_evict(*desc, *cache, keep, recent, workspace,
                            static_cast<cudaStream_t>(stream));
}

}  // extern "C"
