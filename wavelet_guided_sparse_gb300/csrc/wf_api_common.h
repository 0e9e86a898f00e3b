// Argument checks that the entry points of the paged cache and the dense
// attentions share (host side).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "wavefilter.h"
#include "wf_internal.h"

namespace wf {

constexpr size_t kHeaderBytes = 256;  // status word + padding

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

inline int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return WF_OK;
  note_cuda_error(e);
  return WF_ERR_CUDA;
}

inline int check_heads(int q_heads, int kv_heads, int head_dim, int dtype) {
  if (dtype != WF_BF16 && dtype != WF_F32) return WF_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return WF_ERR_UNSUPPORTED;
  if (q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0) return WF_ERR_SHAPE;
  if (q_heads > 65535) return WF_ERR_UNSUPPORTED;  // grid rows
  return WF_OK;
}

inline int check_page_dims(const wf_page_dims* d) {
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
  if ((len / kPagedTile + 1) * d->n_seqs > INT32_MAX) return WF_ERR_UNSUPPORTED;
  return WF_OK;
}

}  // namespace wf
