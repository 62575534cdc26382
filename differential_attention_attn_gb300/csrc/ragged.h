// Launchers of the packed-batch operators (include/diffattn_ragged.h).  Each
// takes validated arguments and enqueues its kernels on `stream`.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/diffattn_ragged.h"
#include "paged.h"

namespace diffattn {

constexpr int64_t kRaggedMaxGroup = 64;

diffattn_status launch_ragged_step(const diffragged_book &book, const int32_t *new_len, int64_t N,
                                   int32_t *q_start, int32_t *positions, int64_t *slots,
                                   int32_t *status, cudaStream_t stream);

diffattn_status launch_ragged_append(const diffattn_desc &desc, const diffpaged_cache &cache,
                                     const void *const src[5], void *const q_out[2],
                                     const diffattn_strides strides[7], const int64_t *slots,
                                     const diffrotary_table *table, const int32_t *positions,
                                     cudaStream_t stream);

// Forward: shares of the work (a CTA at d = 64, a pair of them at d = 128) and workspace offsets.
struct RaggedFwdPlan {
  int32_t shares;
  bool joins;  // a second kernel may have something to do
  size_t part, join, swap;
  size_t bytes;
};
// False when a size does not fit.
bool plan_ragged_fwd(const diffattn_desc &desc, const diffpaged_cache &cache, int sm_count,
                     RaggedFwdPlan *plan);
diffattn_status launch_ragged_fwd(const diffattn_desc &desc, const diffpaged_cache &cache,
                                  const RaggedFwdPlan &plan, const int32_t *q_start, const void *q1,
                                  const void *q2, const float *lambda, const float *norm_w,
                                  void *out, const diffattn_strides strides[3], void *workspace,
                                  cudaStream_t stream);

}  // namespace diffattn
