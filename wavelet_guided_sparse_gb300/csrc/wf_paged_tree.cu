// Attention of drafted trees over a paged cache: dispatch (kernels: wf_paged_umma.cuh,
// and wf_paged_kernel.cuh for few rows and for fp32; plan: wf_paged_window.cu).
#include "wf_paged_umma.cuh"

namespace wf {

cudaError_t launch_paged_tree(const PagedArgs& a, const PagedPlan& plan, cudaStream_t stream) {
  return on_umma(a) ? launch_umma_mask<kMaskTree>(a, plan, stream)
                    : launch_paged_mask<kMaskTree>(a, plan, stream);
}

}  // namespace wf
