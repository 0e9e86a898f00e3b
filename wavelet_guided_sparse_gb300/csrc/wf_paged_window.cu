// Attention of new tokens over a sliding window of a paged cache and its first
// tokens (kernels: wf_paged_kernel.cuh).
#include "wf_paged_kernel.cuh"

namespace wf {

cudaError_t launch_paged_window(const PagedArgs& a, const PagedPlan& plan, cudaStream_t stream) {
  return launch_paged_mask<kMaskWindow>(a, plan, stream);
}

}  // namespace wf
