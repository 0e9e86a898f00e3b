// Attention of drafted trees over a paged cache: plan and dispatch (kernels:
// wf_paged_umma.cuh, and wf_paged_kernel.cuh for few rows and for fp32).
#include "wf_paged_umma.cuh"

namespace wf {

namespace {

// More rows than this a key head run on tcgen05 tiles of 128 rows (bf16; groups
// of up to 128 heads, a node of which fits a tile).  Up to four rows the warps of
// the other kernel add up in one go: four sequences of 300 to 1500 keys 14.6 us
// against 18 there, but 24.8 against 18.9 for 16 rows; 16 sequences of 6800 keys
// 87 against 83.
constexpr int kFewRows = 4;
// What a unit costs its CTA beside its tiles (queries, output, the gap in the
// products), in tiles: about 2 us against 1.6 a tile, 6 with two row tiles.  16
// sequences of 1000 to 16384 keys: 101 -> 95 us.
constexpr int kPadOne = 1, kPadPair = 3;
bool on_umma(const PagedArgs& a) {
  const int g = a.q_heads / a.kv_heads;
  return a.dtype == WF_BF16 && g <= kTileRows && g * a.n_new > kFewRows;
}

}  // namespace

PagedPlan plan_paged_tree(const PagedArgs& a, int sm_count) {
  if (!on_umma(a)) return plan_paged(a, sm_count);
  PagedPlan p;
  const int g = a.q_heads / a.kv_heads, nodes = kTileRows / g;
  p.row_block = a.n_new > nodes ? 2 * nodes * g : kTileRows;
  p.tile = kTileRows;
  p.pad = a.n_new > nodes ? kPadPair : kPadOne;
  const int64_t units = static_cast<int64_t>(a.n_seqs) * a.kv_heads *
                        ((g * a.n_new + p.row_block - 1) / p.row_block);
  const int64_t tiles =
      units * ((static_cast<int64_t>(a.table_pages) * a.page_size + p.tile - 1) / p.tile);
  p.ctas = static_cast<int>(std::min<int64_t>(sm_count, tiles));
  p.part_bytes = static_cast<size_t>(p.ctas) * 2 * p.row_block * (a.head_dim + 2) * sizeof(float);
  return p;
}

cudaError_t launch_paged_tree(const PagedArgs& a, const PagedPlan& plan, cudaStream_t stream) {
  if (!on_umma(a)) return launch_paged_mask<kMaskTree>(a, plan, stream);
  return a.head_dim == 128 ? launch_umma_tree<128>(a, plan, stream)
                           : launch_umma_tree<64>(a, plan, stream);
}

}  // namespace wf
