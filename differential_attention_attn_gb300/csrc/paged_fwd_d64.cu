// diffpaged_fwd's main kernel (paged_fwd.cuh) for d = 64.
#include "paged_fwd.cuh"

namespace diffattn {

diffattn_status launch_paged_main_d64(const FwdParams &p, const CUtensorMap (&maps)[3],
                                      const PagedFwdPlan &plan, bool fp8, cudaStream_t stream) {
  return fp8 ? launch_rows<64, true>(p, maps, plan, stream)
             : launch_rows<64, false>(p, maps, plan, stream);
}

}  // namespace diffattn
