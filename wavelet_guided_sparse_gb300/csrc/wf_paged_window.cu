// Attention of new tokens over a sliding window of a paged cache and its first
// tokens: plan and dispatch (kernels: wf_paged_umma.cuh, and wf_paged_kernel.cuh for
// few rows and for fp32).
#include "wf_paged_umma.cuh"

namespace wf {

PagedPlan plan_paged_masked(const PagedArgs& a, int sm_count) {
  return on_umma(a) ? plan_umma(a, sm_count) : plan_masked(a, sm_count);
}

cudaError_t launch_paged_window(const PagedArgs& a, const PagedPlan& plan, cudaStream_t stream) {
  return on_umma(a) ? launch_umma_mask<kMaskWindow>(a, plan, stream)
                    : launch_paged_mask<kMaskWindow>(a, plan, stream);
}

}  // namespace wf
