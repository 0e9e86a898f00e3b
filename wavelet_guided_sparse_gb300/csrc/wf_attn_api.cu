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
#include "wf_internal.h"

namespace {

constexpr size_t kHeaderBytes = 256;  // status word + padding

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
int elem_bytes(int dtype) { return dtype == WF_BF16 ? 2 : 4; }

int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return WF_OK;
  wf::note_cuda_error(e);
  return WF_ERR_CUDA;
}

int check_heads(int q_heads, int kv_heads, int head_dim, int dtype) {
  if (dtype != WF_BF16 && dtype != WF_F32) return WF_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return WF_ERR_UNSUPPORTED;
  if (q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0) return WF_ERR_SHAPE;
  if (q_heads > 65535) return WF_ERR_UNSUPPORTED;  // grid rows
  return WF_OK;
}

int check_page_dims(const wf_page_dims* d) {
  if (d == nullptr) return WF_ERR_NULL;
  const int st = check_heads(d->q_heads, d->kv_heads, d->head_dim, d->dtype);
  if (st != WF_OK) return st;
  if (d->n_seqs < 1 || d->n_pages < 1 || d->table_pages < 1) return WF_ERR_SHAPE;
  if (d->page_size < 8 || d->page_size > 256 || (d->page_size & (d->page_size - 1)) != 0)
    return WF_ERR_UNSUPPORTED;
  if (d->n_seqs > WF_MAX_SEQS) return WF_ERR_UNSUPPORTED;
  // Cache positions and key tiles are counted in 32 bits, and so are the
  // cache's rows (a tensor copy's row coordinate).
  const int64_t len = static_cast<int64_t>(d->table_pages) * d->page_size;
  const int64_t lines = static_cast<int64_t>(d->n_pages) * d->kv_heads * d->page_size;
  if (len > INT32_MAX - 1024 || lines > INT32_MAX) return WF_ERR_UNSUPPORTED;
  if ((len / wf::kPagedTile + 1) * d->n_seqs > INT32_MAX) return WF_ERR_UNSUPPORTED;
  return WF_OK;
}

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
  const int st = check_page_dims(dims);
  if (st != WF_OK) return st;
  if (bytes == nullptr) return WF_ERR_NULL;
  if (n_new < 1) return WF_ERR_SHAPE;
  if (n_new > WF_MAX_GEN) return WF_ERR_UNSUPPORTED;
  *bytes = kHeaderBytes + wf::plan_paged(paged_args(dims, n_new), wf::device_sm_count()).part_bytes;
  return WF_OK;
}

int wf_paged_attn(const wf_page_dims* dims, const wf_attn_opts* opts, int32_t n_new, const void* Q,
                  const void* K_pages, const void* V_pages, const int32_t* page_table,
                  const int32_t* kv_len, void* O, float* lse, void* workspace,
                  size_t workspace_bytes, void* stream) {
  size_t need = 0;
  int st = wf_paged_attn_workspace_bytes(dims, n_new, &need);
  if (st != WF_OK) return st;
  st = check_opts(opts, dims->head_dim);
  if (st != WF_OK) return st;
  if (Q == nullptr || K_pages == nullptr || V_pages == nullptr || page_table == nullptr ||
      kv_len == nullptr || O == nullptr || workspace == nullptr)
    return WF_ERR_NULL;
  if (!aligned16(Q) || !aligned16(K_pages) || !aligned16(V_pages) || !aligned16(O) ||
      !aligned16(workspace) || !aligned4(page_table) || !aligned4(kv_len) || !aligned4(lse))
    return WF_ERR_ALIGNMENT;
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
  return cuda_status(wf::launch_paged_attn(a, wf::plan_paged(a, wf::device_sm_count()),
                                           static_cast<cudaStream_t>(stream)));
}

int wf_prefill_attn(const wf_prefill_dims* dims, const wf_attn_opts* opts, const void* Q,
                    int64_t q_stride, const void* K, int64_t k_stride, const void* V,
                    int64_t v_stride, const int32_t* cu_q, const int32_t* cu_k, void* O,
                    float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (dims == nullptr) return WF_ERR_NULL;
  int st = check_heads(dims->q_heads, dims->kv_heads, dims->head_dim, dims->dtype);
  if (st != WF_OK) return st;
  if (dims->rows_q < 0 || dims->rows_k < 0 || dims->n_docs < 1) return WF_ERR_SHAPE;
  // Row blocks are counted in 32 bits; rows stay below a grid's limits.
  if (dims->rows_q > (1 << 26) || dims->rows_k > (1 << 30) || dims->n_docs > (1 << 20))
    return WF_ERR_UNSUPPORTED;
  st = check_opts(opts, dims->head_dim);
  if (st != WF_OK) return st;
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
  wf::PrefillArgs a = {};
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
  return cuda_status(wf::launch_prefill(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
