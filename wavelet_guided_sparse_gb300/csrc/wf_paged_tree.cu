// Attention of drafted trees over a paged cache (kernels: wf_paged_kernel.cuh).
#include "wf_paged_kernel.cuh"

namespace wf {

cudaError_t launch_paged_tree(const PagedArgs& a, const PagedPlan& plan, cudaStream_t stream) {
  return launch_paged_mask<kMaskTree>(a, plan, stream);
}

}  // namespace wf
