// C ABI of the paged cache's pages: argument validation, workspace layout and
// dispatch.  Kernels: wf_pages.cu.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "wavefilter.h"
#include "wf_api_common.h"
#include "wf_internal.h"

namespace {

using wf::aligned16;
using wf::aligned4;
using wf::kHeaderBytes;

size_t round16(size_t n) { return (n + 15) & ~static_cast<size_t>(15); }

// Scratch behind the status word: reserve and fork, then (over it) keep.
struct Scratch {
  size_t list, copies, count, alloc_end;  // offsets; base lies at kHeaderBytes
  size_t lines, keep_end;                 // info lies at kHeaderBytes
};
Scratch scratch_of(const wf_page_dims* d, int units, int max_keep, bool fork) {
  Scratch s;
  s.list = kHeaderBytes + round16(sizeof(int32_t) * static_cast<size_t>(units));
  s.copies = s.list + round16(sizeof(int32_t) * static_cast<size_t>(d->n_pages));
  s.count = s.copies + (fork ? sizeof(int4) * static_cast<size_t>(d->n_pages) : 0);
  s.alloc_end = s.count + (fork ? 16 : 0);
  s.lines = kHeaderBytes + sizeof(int4) * static_cast<size_t>(d->n_seqs);
  s.keep_end = s.lines + sizeof(int32_t) * static_cast<size_t>(d->n_seqs) * max_keep;
  return s;
}

// The sizes that matter to pages; query heads do not.
int check_pages(const wf_page_dims* dims, wf_page_dims* d) {
  if (dims == nullptr) return WF_ERR_NULL;
  *d = *dims;
  d->q_heads = d->kv_heads;
  return wf::check_page_dims(d);
}

wf::PagesArgs pages_args(const wf_page_dims& d, int32_t* refs, int32_t* table, void* ws) {
  wf::PagesArgs a = {};
  a.refs = refs;
  a.table = table;
  a.status = static_cast<int32_t*>(ws);
  a.n_seqs = d.n_seqs;
  a.kv_heads = d.kv_heads;
  a.head_dim = d.head_dim;
  a.page_size = d.page_size;
  a.n_pages = d.n_pages;
  a.table_pages = d.table_pages;
  a.dtype = d.dtype;
  return a;
}

// A pool that is named twice (a layer given again, keys that are the values) is taken
// once: two streams would move its rows at the same time.
int check_pools(int n_pools, void* const* pools, bool needed, wf::PagePools* out) {
  out->n = 0;
  if (n_pools < 0 || (needed && n_pools == 0)) return WF_ERR_SHAPE;
  if (n_pools > WF_MAX_POOLS) return WF_ERR_UNSUPPORTED;
  if (n_pools > 0 && pools == nullptr) return WF_ERR_NULL;
  uintptr_t highest = 0;
  for (int i = 0; i < n_pools; ++i) {
    if (pools[i] == nullptr) return WF_ERR_NULL;
    if (!aligned16(pools[i])) return WF_ERR_ALIGNMENT;
    bool again = false;
    if (reinterpret_cast<uintptr_t>(pools[i]) <= highest)
      for (int j = 0; j < out->n; ++j) again |= out->at[j] == pools[i];
    if (again) continue;
    out->at[out->n++] = pools[i];
    highest = std::max(highest, reinterpret_cast<uintptr_t>(pools[i]));
  }
  return WF_OK;
}

template <typename T>
T* at(void* ws, size_t offset) {
  return reinterpret_cast<T*>(static_cast<unsigned char*>(ws) + offset);
}

}  // namespace

extern "C" {

int wf_pages_workspace_bytes(const wf_page_dims* dims, int32_t max_forks, int32_t max_keep,
                             size_t* bytes) {
  wf_page_dims d;
  const int st = check_pages(dims, &d);
  if (st != WF_OK) return st;
  if (bytes == nullptr) return WF_ERR_NULL;
  if (max_forks < 0 || max_keep < 0 || max_keep > d.table_pages * d.page_size) return WF_ERR_SHAPE;
  if (max_forks > WF_MAX_SEQS) return WF_ERR_UNSUPPORTED;
  const Scratch s = scratch_of(&d, std::max(d.n_seqs, max_forks), max_keep, max_forks > 0);
  *bytes = std::max(s.alloc_end, s.keep_end);
  return WF_OK;
}

int wf_paged_reserve(const wf_page_dims* dims, const int32_t* rows, int32_t* refs,
                     int32_t* page_table, void* workspace, size_t workspace_bytes, void* stream) {
  return wf_paged_reserve_from(dims, nullptr, rows, refs, page_table, workspace, workspace_bytes,
                               stream);
}

int wf_paged_reserve_from(const wf_page_dims* dims, const int32_t* from_rows, const int32_t* rows,
                          int32_t* refs, int32_t* page_table, void* workspace,
                          size_t workspace_bytes, void* stream) {
  wf_page_dims d;
  const int st = check_pages(dims, &d);
  if (st != WF_OK) return st;
  if (rows == nullptr || refs == nullptr || page_table == nullptr || workspace == nullptr)
    return WF_ERR_NULL;
  if (!aligned4(from_rows) || !aligned4(rows) || !aligned4(refs) || !aligned4(page_table) ||
      !aligned16(workspace))
    return WF_ERR_ALIGNMENT;
  const Scratch s = scratch_of(&d, d.n_seqs, 0, false);
  if (workspace_bytes < s.alloc_end) return WF_ERR_WORKSPACE;
  wf::AllocArgs x = {};
  x.p = pages_args(d, refs, page_table, workspace);
  x.from = from_rows;
  x.rows = rows;
  x.base = at<int32_t>(workspace, kHeaderBytes);
  x.list = at<int32_t>(workspace, s.list);
  x.units = d.n_seqs;
  return wf::cuda_status(wf::launch_reserve(x, static_cast<cudaStream_t>(stream)));
}

int wf_paged_fork(const wf_page_dims* dims, int32_t n_forks, const int32_t* src,
                  const int32_t* dst, const int32_t* kv_len, const int32_t* share_rows,
                  int32_t* refs, int32_t* page_table, int32_t n_pools, void* const* pools,
                  void* workspace, size_t workspace_bytes, void* stream) {
  wf_page_dims d;
  int st = check_pages(dims, &d);
  if (st != WF_OK) return st;
  if (n_forks < 0) return WF_ERR_SHAPE;
  if (n_forks > WF_MAX_SEQS) return WF_ERR_UNSUPPORTED;
  wf::PagePools p;
  st = check_pools(n_pools, pools, true, &p);
  if (st != WF_OK) return st;
  if (n_forks == 0) return WF_OK;
  if (src == nullptr || dst == nullptr || kv_len == nullptr || refs == nullptr ||
      page_table == nullptr || workspace == nullptr)
    return WF_ERR_NULL;
  if (!aligned4(src) || !aligned4(dst) || !aligned4(kv_len) || !aligned4(share_rows) ||
      !aligned4(refs) || !aligned4(page_table) || !aligned16(workspace))
    return WF_ERR_ALIGNMENT;
  const Scratch s = scratch_of(&d, std::max(d.n_seqs, n_forks), 0, true);
  if (workspace_bytes < s.alloc_end) return WF_ERR_WORKSPACE;
  wf::AllocArgs x = {};
  x.p = pages_args(d, refs, page_table, workspace);
  x.rows = kv_len;
  x.src = src;
  x.dst = dst;
  x.share = share_rows;
  x.base = at<int32_t>(workspace, kHeaderBytes);
  x.list = at<int32_t>(workspace, s.list);
  x.copies = at<int4>(workspace, s.copies);
  x.n_copies = at<int32_t>(workspace, s.count);
  x.units = n_forks;
  return wf::cuda_status(wf::launch_fork(x, p, static_cast<cudaStream_t>(stream)));
}

int wf_paged_keep(const wf_page_dims* dims, const int32_t* kv_len, const int32_t* start,
                  const int32_t* keep, int32_t max_keep, const int32_t* n_keep, int32_t* refs,
                  int32_t* page_table, int32_t n_pools, void* const* pools, void* workspace,
                  size_t workspace_bytes, void* stream) {
  wf_page_dims d;
  int st = check_pages(dims, &d);
  if (st != WF_OK) return st;
  if (max_keep < 0 || max_keep > d.table_pages * d.page_size) return WF_ERR_SHAPE;
  wf::PagePools p;
  st = check_pools(n_pools, pools, keep != nullptr && max_keep > 0, &p);
  if (st != WF_OK) return st;
  if (kv_len == nullptr || start == nullptr || (keep == nullptr) != (n_keep == nullptr) ||
      (keep == nullptr && refs == nullptr) || page_table == nullptr || workspace == nullptr)
    return WF_ERR_NULL;
  if (!aligned4(kv_len) || !aligned4(start) || !aligned4(keep) || !aligned4(n_keep) ||
      !aligned4(refs) || !aligned4(page_table) || !aligned16(workspace))
    return WF_ERR_ALIGNMENT;
  if (keep == nullptr) max_keep = 0;
  const Scratch s = scratch_of(&d, d.n_seqs, max_keep, false);
  if (workspace_bytes < s.keep_end) return WF_ERR_WORKSPACE;
  wf::KeepArgs x = {};
  x.p = pages_args(d, refs, page_table, workspace);
  x.kv_len = kv_len;
  x.start = start;
  x.keep = keep;
  x.n_keep = n_keep;
  x.info = at<int4>(workspace, kHeaderBytes);
  x.lines = at<int32_t>(workspace, s.lines);
  x.max_keep = max_keep;
  return wf::cuda_status(wf::launch_keep(x, p, static_cast<cudaStream_t>(stream)));
}

int wf_paged_release(const wf_page_dims* dims, const int32_t* first, const int32_t* end,
                     int32_t* refs, int32_t* page_table, void* workspace, size_t workspace_bytes,
                     void* stream) {
  wf_page_dims d;
  const int st = check_pages(dims, &d);
  if (st != WF_OK) return st;
  if (first == nullptr || end == nullptr || refs == nullptr || page_table == nullptr)
    return WF_ERR_NULL;
  if (!aligned4(first) || !aligned4(end) || !aligned4(refs) || !aligned4(page_table) ||
      !aligned16(workspace))
    return WF_ERR_ALIGNMENT;
  if (workspace != nullptr && workspace_bytes < kHeaderBytes) return WF_ERR_WORKSPACE;
  return wf::cuda_status(wf::launch_release(pages_args(d, refs, page_table, workspace), first, end,
                                            static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
