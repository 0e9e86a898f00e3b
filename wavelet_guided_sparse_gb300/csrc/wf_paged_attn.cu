// Attention of new tokens over a paged key-value cache: plan and dispatch.
#include <algorithm>

#include "wf_attn.cuh"

namespace wf {

PagedPlan plan_paged(const PagedArgs& a, int sm_count) {
  PagedPlan p;
  const int rows = a.q_heads / a.kv_heads * a.n_new;
  p.row_block = rows <= 16 ? 16 : 64;
  const int64_t units = static_cast<int64_t>(a.n_seqs) * a.kv_heads *
                        ((rows + p.row_block - 1) / p.row_block);
  const int64_t tiles =
      units * ((static_cast<int64_t>(a.table_pages) * a.page_size + kPagedTile - 1) / kPagedTile);
  p.ctas = static_cast<int>(std::min<int64_t>(sm_count * (p.row_block == 16 ? 2 : 1), tiles));
  p.part_bytes = static_cast<size_t>(p.ctas) * 2 * p.row_block * (a.head_dim + 2) * sizeof(float);
  return p;
}

cudaError_t launch_paged_attn(const PagedArgs& a, const PagedPlan& plan, cudaStream_t stream) {
  const cudaError_t e = launch_paged_fma(a, plan, stream);
  if (e != cudaSuccess) return e;
  return launch_paged_join(a, plan, kPagedTile, stream);
}

}  // namespace wf
