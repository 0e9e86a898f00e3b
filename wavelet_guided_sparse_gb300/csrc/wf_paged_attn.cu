// Attention of new tokens over a whole paged cache: plan and dispatch (kernels:
// wf_paged_kernel.cuh).
#include "wf_paged_kernel.cuh"

namespace wf {

PagedPlan plan_paged(const PagedArgs& a, int sm_count) {
  PagedPlan p;
  const int rows = a.q_heads / a.kv_heads * a.n_new;
  p.row_block = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
  p.tile = KT;
  p.pad = 0;
  const int64_t units = static_cast<int64_t>(a.n_seqs) * a.kv_heads *
                        ((rows + p.row_block - 1) / p.row_block);
  const int64_t tiles =
      units * ((static_cast<int64_t>(a.table_pages) * a.page_size + KT - 1) / KT);
  const int per_sm = p.row_block == 16 && a.dtype == WF_BF16 ? 2 : 1;
  p.ctas = static_cast<int>(std::min<int64_t>(sm_count * per_sm, tiles));
  p.part_bytes = static_cast<size_t>(p.ctas) * 2 * p.row_block * (a.head_dim + 2) * sizeof(float);
  return p;
}

cudaError_t launch_paged_attn(const PagedArgs& a, const PagedPlan& plan, cudaStream_t stream) {
  return launch_paged_mask<kMaskPlain>(a, plan, stream);
}

}  // namespace wf
