// Attention over packed sequences: dispatch.
#include "wf_attn.cuh"

namespace wf {

cudaError_t launch_prefill(const PrefillArgs& a, cudaStream_t stream) {
  return launch_prefill_fma(a, stream);
}

}  // namespace wf
