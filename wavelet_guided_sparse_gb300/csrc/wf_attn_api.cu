// C ABI of the paged cache and the dense attentions: argument validation,
// workspace layout and dispatch.  Kernels: wf_append.cu, wf_paged_attn.cu,
// wf_prefill.cu (bf16) and wf_attn_fma.cu (fp32).
//
// As everywhere in this library every entry point validates on the host
// first, enqueues nothing on a validation error, and neither allocates nor
// synchronises.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "wavefilter.h"
#include "wf_api_common.h"
#include "wf_internal.h"

namespace {

using wf::aligned16;
using wf::aligned4;
using wf::check_heads;
using wf::check_page_dims;
using wf::cuda_status;
using wf::kHeaderBytes;

int elem_bytes(int dtype) { return dtype == WF_BF16 ? 2 : 4; }

// Row stride of a [rows, heads, d] operand in elements: whole 16-byte
// chunks, and rows that do not overlap.
bool bad_stride(int64_t stride, int heads, int head_dim, int dtype) {
  return stride < static_cast<int64_t>(heads) * head_dim ||
         stride * elem_bytes(dtype) % 16 != 0 || stride > (int64_t{1} << 36);
}

float scale_of(const wf_attn_opts* o, int head_dim) {
  return o->scale != 0.f ? o->scale : 1.f / std::sqrt(static_cast<float>(head_dim));
}

int check_opts(const wf_attn_opts* o, int head_dim) {
  if (o == nullptr) return WF_ERR_NULL;
  if (!std::isfinite(o->scale) || !std::isfinite(o->softcap) || o->scale < 0.f || o->softcap < 0.f)
    return WF_ERR_SHAPE;
  // As the kernels take them: in the log2 domain, the scale over the cap.
  constexpr float kLog2e = 1.4426950408889634f;
  if (!std::isfinite(o->scale * kLog2e) || !std::isfinite(o->softcap * kLog2e) ||
      (o->softcap > 0.f && (!std::isfinite(std::max(o->scale, 1.f) / o->softcap) ||
                            !std::isnormal(scale_of(o, head_dim) / o->softcap))))
    return WF_ERR_SHAPE;
  if (!aligned4(o->prefix) || !aligned4(o->slopes)) return WF_ERR_ALIGNMENT;
  return WF_OK;
}

// |y| mod 1 as a 64-bit binary fraction, cut; what was cut is added to *below
// in units of its last place.
uint64_t fraction_bits(double y, double* below) {
  y = std::fabs(y);
  const double f = (y - std::floor(y)) * 0x1p64, cut = std::floor(f);
  *below += f - cut;
  return static_cast<uint64_t>(cut);
}

// x / 2 pi mod 1 as a 64-bit binary fraction, to about half its last place for
// |x| up to 2^40.  The quotient is the sum of two doubles, formed with 2 pi as
// the sum of three: positions multiply its error, so that one double's (2^-56
// at x = 1) would show at far positions and high frequencies.
uint64_t turn_fraction(double x) {
  constexpr double kTwoPi[3] = {0x1.921fb54442d18p+2, 0x1.1a62633145c07p-52, -0x1.f1976b7ed8fbcp-108};
  const double y = std::fabs(x), hi = y / kTwoPi[0];
  // What hi leaves of y; the first step is exact.
  const double rest = std::fma(-hi, kTwoPi[1], std::fma(-hi, kTwoPi[0], y)) - hi * kTwoPi[2];
  const double lo = rest / kTwoPi[0];
  double below = 0.0, minus = 0.0;
  uint64_t bits = fraction_bits(hi, &below);
  if (lo < 0.0) {
    bits -= fraction_bits(lo, &minus);
  } else {
    bits += fraction_bits(lo, &below);
  }
  bits += static_cast<uint64_t>(std::llround(below - minus));
  return x < 0.0 ? 0 - bits : bits;
}

wf::PagedArgs paged_args(const wf_page_dims* d, int n_new) {
  wf::PagedArgs a = {};
  a.n_seqs = d->n_seqs;
  a.n_new = n_new;
  a.q_heads = d->q_heads;
  a.kv_heads = d->kv_heads;
  a.head_dim = d->head_dim;
  a.page_size = d->page_size;
  a.n_pages = d->n_pages;
  a.table_pages = d->table_pages;
  a.dtype = d->dtype;
  return a;
}

using PlanFn = wf::PagedPlan (*)(const wf::PagedArgs&, int);

int paged_bytes(const wf_page_dims* dims, int32_t n_new, PlanFn plan, size_t* bytes) {
  const int st = check_page_dims(dims);
  if (st != WF_OK) return st;
  if (bytes == nullptr) return WF_ERR_NULL;
  if (n_new < 1) return WF_ERR_SHAPE;
  if (n_new > WF_MAX_GEN) return WF_ERR_UNSUPPORTED;
  *bytes = kHeaderBytes + plan(paged_args(dims, n_new), wf::device_sm_count()).part_bytes;
  return WF_OK;
}

// What the paged attentions check and hand over alike.
int paged_call(PlanFn plan, const wf_page_dims* dims, const wf_attn_opts* opts, int32_t n_new,
               const void* Q, const void* K_pages, const void* V_pages, const int32_t* page_table,
               const int32_t* kv_len, void* O, float* lse, void* workspace, size_t workspace_bytes,
               wf::PagedArgs* out) {
  size_t need = 0;
  int st = paged_bytes(dims, n_new, plan, &need);
  if (st != WF_OK) return st;
  st = check_opts(opts, dims->head_dim);
  if (st != WF_OK) return st;
  if (Q == nullptr || K_pages == nullptr || V_pages == nullptr || page_table == nullptr ||
      kv_len == nullptr || O == nullptr || workspace == nullptr)
    return WF_ERR_NULL;
  if (!aligned16(Q) || !aligned16(K_pages) || !aligned16(V_pages) || !aligned16(O) ||
      !aligned16(workspace) || !aligned4(page_table) || !aligned4(kv_len) || !aligned4(lse))
    return WF_ERR_ALIGNMENT;
  // Tiles of all sequences, with the empty ones behind a unit's, are counted in 32 bits.
  const wf::PagedPlan p = plan(paged_args(dims, n_new), wf::device_sm_count());
  const int64_t len = static_cast<int64_t>(dims->table_pages) * dims->page_size;
  if (((len + p.tile - 1) / p.tile + p.pad) * dims->n_seqs > INT32_MAX) return WF_ERR_UNSUPPORTED;
  if (workspace_bytes < need) return WF_ERR_WORKSPACE;
  wf::PagedArgs a = paged_args(dims, n_new);
  a.q = Q;
  a.k_pages = K_pages;
  a.v_pages = V_pages;
  a.table = page_table;
  a.kv_len = kv_len;
  a.o = O;
  a.lse = lse;
  a.status = static_cast<int32_t*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + kHeaderBytes);
  a.scale = scale_of(opts, dims->head_dim);
  a.softcap = opts->softcap;
  a.causal = opts->causal != 0;
  a.prefix = opts->prefix;
  a.slopes = opts->slopes;
  *out = a;
  return WF_OK;
}

int check_window(const wf_attn_opts* opts, int32_t window, int32_t sinks) {
  if (window < 1 || sinks < 0) return WF_ERR_SHAPE;
  return opts != nullptr && opts->prefix != nullptr ? WF_ERR_UNSUPPORTED : WF_OK;
}

// What the packed-prompt attentions check and hand over alike; *out has no rows
// where there is nothing to do.
int prefill_call(const wf_prefill_dims* dims, const wf_attn_opts* opts, const void* Q,
                 int64_t q_stride, const void* K, int64_t k_stride, const void* V, int64_t v_stride,
                 const int32_t* cu_q, const int32_t* cu_k, void* O, float* lse, void* workspace,
                 size_t workspace_bytes, wf::PrefillArgs* out) {
  if (dims == nullptr) return WF_ERR_NULL;
  int st = check_heads(dims->q_heads, dims->kv_heads, dims->head_dim, dims->dtype);
  if (st != WF_OK) return st;
  if (dims->rows_q < 0 || dims->rows_k < 0 || dims->n_docs < 1) return WF_ERR_SHAPE;
  // Row blocks are counted in 32 bits; rows stay below a grid's limits.
  if (dims->rows_q > (1 << 26) || dims->rows_k > (1 << 30) || dims->n_docs > (1 << 20))
    return WF_ERR_UNSUPPORTED;
  st = check_opts(opts, dims->head_dim);
  if (st != WF_OK) return st;
  *out = wf::PrefillArgs{};
  if (dims->rows_q == 0) return WF_OK;
  if (Q == nullptr || cu_q == nullptr || cu_k == nullptr || O == nullptr ||
      (dims->rows_k > 0 && (K == nullptr || V == nullptr)))
    return WF_ERR_NULL;
  if (bad_stride(q_stride, dims->q_heads, dims->head_dim, dims->dtype) ||
      bad_stride(k_stride, dims->kv_heads, dims->head_dim, dims->dtype) ||
      bad_stride(v_stride, dims->kv_heads, dims->head_dim, dims->dtype))
    return WF_ERR_SHAPE;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O) || !aligned16(workspace) ||
      !aligned4(cu_q) || !aligned4(cu_k) || !aligned4(lse))
    return WF_ERR_ALIGNMENT;
  if (workspace != nullptr && workspace_bytes < kHeaderBytes) return WF_ERR_WORKSPACE;
  wf::PrefillArgs& a = *out;
  a.q = Q;
  a.k = K;
  a.v = V;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.o = O;
  a.lse = lse;
  a.status = static_cast<int32_t*>(workspace);
  a.rows_q = dims->rows_q;
  a.rows_k = dims->rows_k;
  a.n_docs = dims->n_docs;
  a.q_heads = dims->q_heads;
  a.kv_heads = dims->kv_heads;
  a.head_dim = dims->head_dim;
  a.dtype = dims->dtype;
  a.scale = scale_of(opts, dims->head_dim);
  a.softcap = opts->softcap;
  a.causal = opts->causal != 0;
  a.prefix = opts->prefix;
  a.slopes = opts->slopes;
  return WF_OK;
}

}  // namespace

extern "C" {

int wf_rope_inv_freq(int32_t rotary_dim, double base, double* out) {
  if (out == nullptr) return WF_ERR_NULL;
  if (rotary_dim < 16 || rotary_dim > 128 || rotary_dim % 16 != 0 || !(base > 1.0) ||
      !std::isfinite(base))
    return WF_ERR_UNSUPPORTED;
  for (int i = 0; i < rotary_dim / 2; ++i) out[i] = std::pow(base, -2.0 * i / rotary_dim);
  return WF_OK;
}

int wf_paged_append(const wf_page_dims* dims, int32_t n_rows, const void* Q, int64_t q_stride,
                    const void* K, int64_t k_stride, const void* V, int64_t v_stride,
                    const int32_t* cu_rows, const int32_t* cache_len, const int32_t* positions,
                    const int32_t* page_table, const double* inv_freq, int32_t rotary_dim,
                    int32_t interleaved, void* K_pages, void* V_pages, void* Q_out, void* K_out,
                    void* workspace, size_t workspace_bytes, void* stream) {
  const int st = check_page_dims(dims);
  if (st != WF_OK) return st;
  if (n_rows < 0 || rotary_dim < 0 || rotary_dim > dims->head_dim || rotary_dim % 16 != 0)
    return WF_ERR_SHAPE;
  if (n_rows == 0) return WF_OK;
  if (K == nullptr || V == nullptr || cu_rows == nullptr || cache_len == nullptr ||
      page_table == nullptr || K_pages == nullptr || V_pages == nullptr ||
      (Q == nullptr) != (Q_out == nullptr) || (rotary_dim > 0 && inv_freq == nullptr))
    return WF_ERR_NULL;
  if ((Q != nullptr && bad_stride(q_stride, dims->q_heads, dims->head_dim, dims->dtype)) ||
      bad_stride(k_stride, dims->kv_heads, dims->head_dim, dims->dtype) ||
      bad_stride(v_stride, dims->kv_heads, dims->head_dim, dims->dtype))
    return WF_ERR_SHAPE;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(K_pages) ||
      !aligned16(V_pages) || !aligned16(Q_out) || !aligned16(K_out) || !aligned16(workspace) ||
      !aligned4(cu_rows) || !aligned4(cache_len) || !aligned4(positions) || !aligned4(page_table))
    return WF_ERR_ALIGNMENT;
  if (workspace != nullptr && workspace_bytes < kHeaderBytes) return WF_ERR_WORKSPACE;
  wf::RopeTurns turns = {};
  for (int i = 0; i < rotary_dim / 2; ++i) {
    if (!std::isfinite(inv_freq[i])) return WF_ERR_SHAPE;
    turns.f[i] = turn_fraction(inv_freq[i]);
  }
  wf::AppendArgs a = {};
  a.q = Q;
  a.k = K;
  a.v = V;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.cu_rows = cu_rows;
  a.cache_len = cache_len;
  a.positions = positions;
  a.table = page_table;
  a.k_pages = K_pages;
  a.v_pages = V_pages;
  a.q_out = Q_out;
  a.k_out = K_out;
  a.status = static_cast<int32_t*>(workspace);
  a.rows = n_rows;
  a.n_seqs = dims->n_seqs;
  a.q_heads = dims->q_heads;
  a.kv_heads = dims->kv_heads;
  a.head_dim = dims->head_dim;
  a.page_size = dims->page_size;
  a.n_pages = dims->n_pages;
  a.table_pages = dims->table_pages;
  a.dtype = dims->dtype;
  a.rotary_dim = rotary_dim;
  a.interleaved = interleaved != 0;
  return cuda_status(wf::launch_append(a, turns, static_cast<cudaStream_t>(stream)));
}

int wf_paged_attn_workspace_bytes(const wf_page_dims* dims, int32_t n_new, size_t* bytes) {
  return paged_bytes(dims, n_new, wf::plan_paged, bytes);
}

int wf_paged_attn(const wf_page_dims* dims, const wf_attn_opts* opts, int32_t n_new, const void* Q,
                  const void* K_pages, const void* V_pages, const int32_t* page_table,
                  const int32_t* kv_len, void* O, float* lse, void* workspace,
                  size_t workspace_bytes, void* stream) {
  wf::PagedArgs a;
  const int st = paged_call(wf::plan_paged, dims, opts, n_new, Q, K_pages, V_pages, page_table,
                            kv_len, O, lse, workspace, workspace_bytes, &a);
  if (st != WF_OK) return st;
  return cuda_status(wf::launch_paged_attn(a, wf::plan_paged(a, wf::device_sm_count()),
                                           static_cast<cudaStream_t>(stream)));
}

int wf_paged_window_attn(const wf_page_dims* dims, const wf_attn_opts* opts, int32_t window,
                         int32_t sinks, int32_t n_new, const void* Q, const void* K_pages,
                         const void* V_pages, const int32_t* page_table, const int32_t* kv_len,
                         void* O, float* lse, void* workspace, size_t workspace_bytes,
                         void* stream) {
  wf::PagedArgs a;
  int st = check_window(opts, window, sinks);
  if (st != WF_OK) return st;
  st = paged_call(wf::plan_paged_masked, dims, opts, n_new, Q, K_pages, V_pages, page_table, kv_len,
                  O, lse, workspace, workspace_bytes, &a);
  if (st != WF_OK) return st;
  // So large a window hides nothing; positions minus it stay within 32 bits.
  a.window = std::min(window, INT32_MAX - 512);
  a.sinks = sinks;
  return cuda_status(wf::launch_paged_window(a, wf::plan_paged_masked(a, wf::device_sm_count()),
                                             static_cast<cudaStream_t>(stream)));
}

int wf_paged_window_attn_workspace_bytes(const wf_page_dims* dims, int32_t n_new, size_t* bytes) {
  return paged_bytes(dims, n_new, wf::plan_paged_masked, bytes);
}

int wf_paged_tree_attn_workspace_bytes(const wf_page_dims* dims, int32_t n_nodes, size_t* bytes) {
  return paged_bytes(dims, n_nodes, wf::plan_paged_masked, bytes);
}

int wf_paged_tree_attn(const wf_page_dims* dims, const wf_attn_opts* opts, int32_t n_nodes,
                       const void* Q, const void* K_pages, const void* V_pages,
                       const int32_t* page_table, const int32_t* kv_len, const int32_t* parents,
                       const int32_t* tree_len, void* O, float* lse, void* workspace,
                       size_t workspace_bytes, void* stream) {
  if (opts != nullptr && (opts->causal == 0 || opts->prefix != nullptr)) return WF_ERR_UNSUPPORTED;
  wf::PagedArgs a;
  const int st = paged_call(wf::plan_paged_masked, dims, opts, n_nodes, Q, K_pages, V_pages,
                            page_table, kv_len, O, lse, workspace, workspace_bytes, &a);
  if (st != WF_OK) return st;
  if (parents == nullptr) return WF_ERR_NULL;
  if (!aligned4(parents) || !aligned4(tree_len)) return WF_ERR_ALIGNMENT;
  a.parents = parents;
  a.tree_len = tree_len;
  return cuda_status(wf::launch_paged_tree(a, wf::plan_paged_masked(a, wf::device_sm_count()),
                                           static_cast<cudaStream_t>(stream)));
}

int wf_prefill_attn(const wf_prefill_dims* dims, const wf_attn_opts* opts, const void* Q,
                    int64_t q_stride, const void* K, int64_t k_stride, const void* V,
                    int64_t v_stride, const int32_t* cu_q, const int32_t* cu_k, void* O,
                    float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  wf::PrefillArgs a;
  const int st = prefill_call(dims, opts, Q, q_stride, K, k_stride, V, v_stride, cu_q, cu_k, O, lse,
                              workspace, workspace_bytes, &a);
  if (st != WF_OK || a.rows_q == 0) return st;
  return cuda_status(wf::launch_prefill(a, static_cast<cudaStream_t>(stream)));
}

int wf_prefill_window_attn(const wf_prefill_dims* dims, const wf_attn_opts* opts, int32_t window,
                           int32_t sinks, const void* Q, int64_t q_stride, const void* K,
                           int64_t k_stride, const void* V, int64_t v_stride, const int32_t* cu_q,
                           const int32_t* cu_k, void* O, float* lse, void* workspace,
                           size_t workspace_bytes, void* stream) {
  int st = check_window(opts, window, sinks);
  if (st != WF_OK) return st;
  wf::PrefillArgs a;
  st = prefill_call(dims, opts, Q, q_stride, K, k_stride, V, v_stride, cu_q, cu_k, O, lse,
                    workspace, workspace_bytes, &a);
  if (st != WF_OK || a.rows_q == 0) return st;
  // So large a window hides nothing (positions lie in [-2^26, 2^30)).
  a.window = std::min(window, (1 << 30) + (1 << 26) + 1);
  a.sinks = sinks;
  return cuda_status(wf::launch_prefill(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
