// C ABI of the packed-batch operators: argument validation and dispatch.  Every
// entry point is declared, with its contract, in include/diffattn_ragged.h.
#include <cuda_runtime.h>

#include <cstdint>

#include "ragged.h"
#include "rotary.cuh"

using namespace diffattn;

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The token and head strides of a packed tensor.
bool packed_strides_ok(const diffattn_strides &s, int64_t multiple) {
  return paged_strides_ok({multiple, s.h, s.n}, multiple);
}

// Everything about a forward but its tensors, without a device.
diffattn_status check_fwd(const diffattn_desc *desc, const diffpaged_cache *cache) {
  const diffattn_status st = check_paged_cache(desc, cache, true);
  if (st != DIFFATTN_OK) return st;
  if (desc->H / cache->kv_heads > kRaggedMaxGroup || desc->N > (int64_t{1} << 30) ||
      desc->B >= (int64_t{1} << 24) || desc->H > 65535)
    return DIFFATTN_ERR_UNSUPPORTED;
  if (desc->B == 0 || desc->H == 0 || desc->N == 0) return DIFFATTN_OK;
  RaggedFwdPlan plan;
  return plan_ragged_fwd(*desc, *cache, 2, &plan) ? DIFFATTN_OK : DIFFATTN_ERR_UNSUPPORTED;
}

diffattn_status plan_fwd(const diffattn_desc &desc, const diffpaged_cache &cache,
                         RaggedFwdPlan *plan) {
  *plan = RaggedFwdPlan{};
  if (desc.B == 0 || desc.H == 0 || desc.N == 0) return DIFFATTN_OK;
  const int sms = device_sm_count();
  if (sms <= 1) return DIFFATTN_ERR_CUDA;
  return plan_ragged_fwd(desc, cache, sms, plan) ? DIFFATTN_OK : DIFFATTN_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" {

diffattn_status diffragged_step(const diffragged_book *book, const int32_t *new_len, int64_t N,
                                int32_t *q_start, int32_t *positions, int64_t *slots,
                                int32_t *status, void *stream) {
  if (book == nullptr || N < 0) return DIFFATTN_ERR_INVALID_ARG;
  if (book->B < 0 || book->max_pages < 1 || book->capacity < 0 || book->page_size < 1 ||
      book->reserved != 0)
    return DIFFATTN_ERR_INVALID_ARG;
  if (book->B >= (int64_t{1} << 24) || book->max_pages >= (int64_t{1} << 30) / book->page_size ||
      book->capacity > (int64_t{1} << 30) || N > (int64_t{1} << 30))
    return DIFFATTN_ERR_UNSUPPORTED;
  if (q_start == nullptr || !aligned(q_start, 4) || !aligned(positions, 4) || !aligned(slots, 8) ||
      !aligned(status, 4))
    return DIFFATTN_ERR_INVALID_ARG;
  if (book->B > 0) {
    if (!book->kv_len || !book->held || !book->page_table || !book->free_count || !new_len ||
        (book->capacity > 0 && !book->free_pages))
      return DIFFATTN_ERR_INVALID_ARG;
    for (const void *x : {static_cast<const void *>(book->kv_len),
                          static_cast<const void *>(book->held),
                          static_cast<const void *>(book->page_table),
                          static_cast<const void *>(book->free_pages),
                          static_cast<const void *>(book->free_count),
                          static_cast<const void *>(new_len)})
      if (!aligned(x, 4)) return DIFFATTN_ERR_INVALID_ARG;
  } else if (book->free_count == nullptr || !aligned(book->free_count, 4)) {
    return DIFFATTN_ERR_INVALID_ARG;
  }
  const diffattn_status st = require_sm103();
  if (st != DIFFATTN_OK) return st;
  return launch_ragged_step(*book, new_len, N, q_start, positions, slots, status,
                            static_cast<cudaStream_t>(stream));
}

diffattn_status diffragged_append(const diffattn_desc *desc, const diffpaged_cache *cache,
                                  const void *q1, const void *q2, const void *k1, const void *k2,
                                  const void *v, void *q1_out, void *q2_out,
                                  const diffattn_strides *strides, const int64_t *slots,
                                  const diffrotary_table *table, const int32_t *positions,
                                  void *stream) {
  diffattn_status st = check_paged_cache(desc, cache, true);
  if (st != DIFFATTN_OK) return st;
  if (table != nullptr && !rotary_table_ok(*table, desc->d)) return DIFFATTN_ERR_INVALID_ARG;
  const bool q = q1 != nullptr;
  if (q != (q2 != nullptr) || q != (q1_out != nullptr) || q != (q2_out != nullptr))
    return DIFFATTN_ERR_INVALID_ARG;
  const int64_t d = desc->d, H = desc->H, kv = cache->kv_heads;
  if (desc->N == 0 || desc->B == 0 || H == 0) return DIFFATTN_OK;
  if (!k1 || !k2 || !v || !slots || !aligned(slots, 8) || (table && !positions) ||
      !aligned(positions, 4))
    return DIFFATTN_ERR_INVALID_ARG;
  for (const void *x : {q1, q2, k1, k2, v, static_cast<const void *>(q1_out),
                        static_cast<const void *>(q2_out)})
    if (!aligned(x, 16)) return DIFFATTN_ERR_INVALID_ARG;
  const bool fp8 = desc->dtype == DIFFATTN_E4M3_QK;
  diffattn_strides st7[7];
  for (int i = 0; i < 7; ++i) {
    const int64_t heads = i == 2 || i == 3 || i == 4 ? kv : H, width = i == 4 ? 2 * d : d;
    st7[i] = strides ? strides[i] : diffattn_strides{0, width, heads * width};
    if ((q || (i >= 2 && i < 5)) && !packed_strides_ok(st7[i], fp8 && i >= 5 ? 16 : 8))
      return DIFFATTN_ERR_INVALID_ARG;
  }
  for (int i = 0; i < 2; ++i) {
    const void *in = i ? q2 : q1, *out = i ? q2_out : q1_out;
    if (q && in == out && (fp8 || st7[i].h != st7[5 + i].h || st7[i].n != st7[5 + i].n))
      return DIFFATTN_ERR_INVALID_ARG;
  }
  // (The kernel's blocks: 16 tokens and a head each at least.)
  if (desc->N > (int64_t{1} << 30) || 2 * H + 4 * kv > 65535 ||
      (desc->N / 16 + 1) * (2 * H + 4 * kv) >= (int64_t{1} << 31))
    return DIFFATTN_ERR_UNSUPPORTED;
  if ((st = require_sm103()) != DIFFATTN_OK) return st;
  const void *const src[5] = {q1, q2, k1, k2, v};
  void *const out[2] = {q1_out, q2_out};
  return launch_ragged_append(*desc, *cache, src, out, st7, slots, table, positions,
                              static_cast<cudaStream_t>(stream));
}

diffattn_status diffragged_fwd_plan(const diffattn_desc *desc, const diffpaged_cache *cache,
                                    size_t *workspace_bytes) {
  if (workspace_bytes == nullptr) return DIFFATTN_ERR_INVALID_ARG;
  RaggedFwdPlan plan;
  diffattn_status st = check_fwd(desc, cache);
  if (st == DIFFATTN_OK) st = plan_fwd(*desc, *cache, &plan);
  if (st == DIFFATTN_OK) *workspace_bytes = plan.bytes;
  return st;
}

diffattn_status diffragged_fwd(const diffattn_desc *desc, const diffpaged_cache *cache,
                               const int32_t *q_start, const void *q1, const void *q2,
                               const float *lambda, const float *norm_w, void *out,
                               const diffattn_strides *strides, void *workspace,
                               size_t workspace_bytes, void *stream) {
  diffattn_status st = check_fwd(desc, cache);
  if (st != DIFFATTN_OK) return st;
  if (desc->B == 0 || desc->H == 0 || desc->N == 0) return DIFFATTN_OK;
  if (!q_start || !q1 || !q2 || !lambda || !out || !aligned(q_start, 4) || !aligned(q1, 16) ||
      !aligned(q2, 16) || !aligned(out, 16) || !aligned(lambda, 4) || !aligned(norm_w, 16))
    return DIFFATTN_ERR_INVALID_ARG;
  const bool fp8 = desc->dtype == DIFFATTN_E4M3_QK;
  diffattn_strides st3[3];
  for (int i = 0; i < 3; ++i) {
    const int64_t width = i == 2 ? 2 * desc->d : desc->d;
    st3[i] = strides ? strides[i] : diffattn_strides{0, width, desc->H * width};
    if (!packed_strides_ok(st3[i], fp8 && i < 2 ? 16 : 8)) return DIFFATTN_ERR_INVALID_ARG;
  }
  RaggedFwdPlan plan;
  if ((st = plan_fwd(*desc, *cache, &plan)) != DIFFATTN_OK) return st;
  if (plan.bytes > 0 &&
      (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < plan.bytes))
    return DIFFATTN_ERR_INVALID_ARG;
  if ((st = require_sm103()) != DIFFATTN_OK) return st;
  return launch_ragged_fwd(*desc, *cache, plan, q_start, q1, q2, lambda, norm_w, out, st3, workspace,
                           static_cast<cudaStream_t>(stream));
}

}  // extern "C"
