// The pages of a paged cache: taking free ones, sharing and copying them,
// moving kept rows together, giving them back.
//
// refs[p] counts the page table entries that hold page p; a page with 0 is
// free.  Entries without a page are negative; a reserve fills them from a row on (those
// that a window has given back lie below it), a fork leaves them as they are.  Free
// pages are taken lowest first: the i-th entry that needs a page (sequence by sequence,
// entry by entry) gets the i-th lowest free one, so that the result is a function of
// the inputs alone.
//
// alloc_kernel (reserve, fork) counts needs and free pages in one cluster,
// each CTA and warp over a contiguous share of both, exchanges the counts
// through distributed shared memory, lists the free pages by rank and fills
// the entries from that list.  Up to kOneCta pages one CTA does it, its list in
// shared memory (2 us less), above that eight share the pass over refs.
//
// copy_pages_kernel moves what a fork copies: HBM-bound, each warp takes one
// head's rows of a page (contiguous) of one pool and keeps eight 16-byte loads
// a lane in flight.
//
// move_rows_kernel moves kept rows up in place.  Kept rows ascend, so row i
// (destination start + i) never lands on the source of a later one, and a
// group (a warp or a CTA) may read a step's rows, and the next step's, meet,
// and write the first.  Rows are split into 128-byte pieces: each (sequence,
// pool, head, piece) is one independent stream in order.
//
// Measured (8 heads of keys, d = 128, bf16).  Four sequences of 16384 rows copied in
// 4 layers: 338 us with the release, 92 % of the copy rate.  4096 of 32768 rows of
// four sequences moved in 4 layers: 80 us, the copy rate (in one CTA a stream; with
// plan and launches 94).  Small calls are launches and dependent loads: reserve and
// keep of 16 accepted paths in 8 layers 13.5 us, 32 forks of shared pages in 8 layers
// with their release 15.5.
#include <algorithm>

#include "wf_attn.cuh"

namespace wf {

namespace {

constexpr int kAllocThreads = 1024, kAllocWarps = kAllocThreads / 32, kAllocCluster = 8;
constexpr int kOneCta = 16384;  // pages that one CTA counts alone
constexpr int kSeqWords = WF_MAX_SEQS / 32;

// Every kernel here is launched early.
__device__ __forceinline__ int ld(const int32_t* p) { return load_input<kReadOrdered>(p); }

__device__ __forceinline__ int max_len(const PagesArgs& a) { return a.table_pages * a.page_size; }

__device__ __forceinline__ int page_shift(const PagesArgs& a) { return __ffs(a.page_size) - 1; }

// A length clamped into a sequence's table; flags one outside.
__device__ __forceinline__ int length_in(const PagesArgs& a, int n, bool say) {
  if (say && (n < 0 || n > max_len(a))) raise_flag(a.status, WF_DEV_BAD_INDEX);
  return min(max(n, 0), max_len(a));
}

// One reference less; flags a page that had none.
__device__ __forceinline__ void drop_page(const PagesArgs& a, int page) {
  if (page >= a.n_pages || atomicSub(a.refs + page, 1) <= 0) {
    if (page < a.n_pages) atomicAdd(a.refs + page, 1);
    raise_flag(a.status, WF_DEV_BAD_INDEX);
  }
}

// Entries [first, end) of a sequence's table row, by threads thread, thread +
// threads, ...: their pages lose a reference, the entries become -1.
__device__ __forceinline__ void drop_entries(const PagesArgs& a, int s, int first, int end,
                                             int thread, int threads) {
  int32_t* row = a.table + static_cast<int64_t>(s) * a.table_pages;
  for (int e = first + thread; e < end; e += threads) {
    const int page = row[e];
    if (page < 0) continue;
    row[e] = -1;
    drop_page(a, page);
  }
}

// What a fork takes: parent, child, entries that are shared, entries in all.
struct ForkUnit {
  int src, dst, shared, entries, len;
};

constexpr int kBatch = 8;  // loads of a lane that fly together
constexpr int kLocalList = 4096;  // free pages that one CTA lists in shared memory

struct AllocShared {
  uint32_t is_src[kSeqWords], once[kSeqWords], twice[kSeqWords];
  int warp_need[kAllocWarps], warp_free[kAllocWarps];
  int need[kAllocCluster], free[kAllocCluster];  // every CTA's totals
  int list[kLocalList];                          // one CTA: its free pages by rank
};

__device__ __forceinline__ bool bit_of(const uint32_t* words, int i) {
  return (words[i >> 5] >> (i & 31)) & 1;
}

// Fork i, or entries = 0 where it is unsound (a row outside the table, a child
// that is also a parent, or one of two forks).  Entries that a parent has no page for
// (what a window left behind) cost none and stay without one.
__device__ __forceinline__ ForkUnit fork_unit(const AllocArgs& x, const AllocShared& sm, int i,
                                              bool say) {
  const PagesArgs& a = x.p;
  ForkUnit u = {ld(x.src + i), ld(x.dst + i), 0, 0, 0};
  if (static_cast<unsigned>(u.src) >= static_cast<unsigned>(a.n_seqs) ||
      static_cast<unsigned>(u.dst) >= static_cast<unsigned>(a.n_seqs)) {
    if (say) raise_flag(a.status, WF_DEV_BAD_INDEX);
    u.dst = -1;
    return u;
  }
  if (bit_of(sm.is_src, u.dst) || bit_of(sm.twice, u.dst)) {
    if (say) raise_flag(a.status, WF_DEV_DUP_INDEX);
    u.dst = -1;
    return u;
  }
  u.len = length_in(a, ld(x.rows + u.src), say);
  const int shift = page_shift(a);
  u.entries = (u.len + a.page_size - 1) >> shift;
  const int share = x.share != nullptr ? min(max(ld(x.share + i), 0), u.len) : u.len;
  u.shared = share >> shift;
  return u;
}

// Entries [first, end) of sequence s, of which a reserve fills those without a page.
struct ReserveUnit {
  int first, end;
};
template <bool FROM>
__device__ __forceinline__ ReserveUnit reserve_unit(const AllocArgs& x, int s, bool say) {
  const int shift = page_shift(x.p), rows = length_in(x.p, ld(x.rows + s), say);
  ReserveUnit u = {0, (rows + x.p.page_size - 1) >> shift};
  if (FROM) {
    const int from = length_in(x.p, ld(x.from + s), say);
    u.first = from < rows ? from >> shift : u.end;
  }
  return u;
}

// Sums of needs are cut at `most`, one page more than there are: the entries of a call
// may be more than 32 bits count, and behind the last page it does not matter how
// many want one.
__device__ __forceinline__ int sum_cut(int a, int b, int most) { return min(a + b, most); }
// Sums of a warp's values up to each lane's, its own left out; `total`: all.
__device__ __forceinline__ int sums_before(int v, int most, int lane, int* total) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = sum_cut(v, x, most);
  }
  *total = __shfl_sync(0xffffffffu, v, 31);
  const int before = __shfl_up_sync(0xffffffffu, v, 1);
  return lane == 0 ? 0 : before;
}

// Words first + lane, first + 32 + lane, ... of an array that ends at `end`
// (`with` behind it), all loads in flight together.
__device__ __forceinline__ void read_batch(const int32_t* from, int first, int end, int lane,
                                           int with, int (&got)[kBatch]) {
#pragma unroll
  for (int k = 0; k < kBatch; ++k) {
    const int i = first + 32 * k + lane;
    got[k] = i < end ? from[i] : with;
  }
}

// FROM: a reserve with a lower bound of rows (one kernel for both costs each 0.3 us).
template <bool FORK, bool FROM>
__global__ void __launch_bounds__(kAllocThreads) alloc_kernel(const AllocArgs x) {
  __shared__ AllocShared sm;
  const PagesArgs& a = x.p;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = static_cast<int>(cluster.num_blocks());
  const int me = static_cast<int>(cluster.block_rank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gw = me * kAllocWarps + warp, warps = ctas * kAllocWarps;
  launch_dependents();
  wait_for_primary();
  if (FORK) {
    for (int i = threadIdx.x; i < kSeqWords; i += kAllocThreads)
      sm.is_src[i] = sm.once[i] = sm.twice[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < x.units; i += kAllocThreads) {
      const int s = ld(x.src + i), d = ld(x.dst + i);
      if (static_cast<unsigned>(s) < static_cast<unsigned>(a.n_seqs))
        atomicOr(&sm.is_src[s >> 5], 1u << (s & 31));
      if (static_cast<unsigned>(d) < static_cast<unsigned>(a.n_seqs) &&
          (atomicOr(&sm.once[d >> 5], 1u << (d & 31)) >> (d & 31) & 1))
        atomicOr(&sm.twice[d >> 5], 1u << (d & 31));
    }
    __syncthreads();
  }
  // This warp's units and pages, both contiguous in order.
  const int u0 = static_cast<int>(static_cast<int64_t>(x.units) * gw / warps);
  const int u1 = static_cast<int>(static_cast<int64_t>(x.units) * (gw + 1) / warps);
  const int p0 = static_cast<int>(static_cast<int64_t>(a.n_pages) * gw / warps);
  const int p1 = static_cast<int>(static_cast<int64_t>(a.n_pages) * (gw + 1) / warps);
  // This warp's first counts, kept: of a small pool all of them.
  int refs0[kBatch];
  read_batch(a.refs, p0, p1, lane, 1, refs0);
  // What this warp's first unit is, kept too: behind the barriers its words would come
  // from L2 once more.
  const int most = a.n_pages + 1;
  ForkUnit fork0 = {};
  ReserveUnit unit0 = {};
  bool odd = false;  // some child's row holds negative entries that are not -1
  int need = 0;
  for (int u = u0; u < u1; ++u) {
    int more = 0;
    bool skip = false;
    if (FORK) {
      // Both rows' first entries come in beside the parent's length.
      const auto row_of = [&](int s) {
        return a.table + static_cast<int64_t>(min(max(s, 0), a.n_seqs - 1)) * a.table_pages;
      };
      const int32_t *from = row_of(ld(x.src + u)), *to = row_of(ld(x.dst + u));
      int parents[kBatch], children[kBatch];
      read_batch(from, 0, a.table_pages, lane, -1, parents);
      read_batch(to, 0, a.table_pages, lane, -1, children);
      const ForkUnit f = fork_unit(x, sm, u, lane == 0);
      if (u == u0) fork0 = f;
      skip = f.dst < 0;
      bool held = false;
      for (int e0 = 0; e0 < a.table_pages && !skip; e0 += 32 * kBatch) {
        const bool count = e0 < f.entries && e0 + 32 * kBatch > f.shared;
        if (e0 > 0) {
          if (count) read_batch(from, e0, f.entries, lane, -1, parents);
          read_batch(to, e0, a.table_pages, lane, -1, children);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          held |= children[k] >= 0;
          odd |= children[k] < -1;
        }
        if (!count) continue;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int e = e0 + 32 * k + lane;
          more += __popc(
              __ballot_sync(0xffffffffu, parents[k] >= 0 && e >= f.shared && e < f.entries));
        }
      }
      if (__any_sync(0xffffffffu, held)) {  // its references would be lost
        if (lane == 0) raise_flag(a.status, WF_DEV_BAD_INDEX);
        skip = true;
        more = 0;
      }
    } else {
      const ReserveUnit r = reserve_unit<FROM>(x, u, lane == 0);
      if (u == u0) unit0 = r;
      const int32_t* row = a.table + static_cast<int64_t>(u) * a.table_pages;
      for (int e0 = r.first; e0 < r.end; e0 += 32 * kBatch) {
        int got[kBatch];
        read_batch(row, e0, r.end, lane, 0, got);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) more += __popc(__ballot_sync(0xffffffffu, got[k] < 0));
      }
    }
    if (lane == 0) x.base[u] = skip ? -1 : need;  // within the warp
    need = sum_cut(need, more, most);
  }
  int free = 0;
  for (int p = p0; p < p1; p += 32 * kBatch) {
    int got[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) got[k] = refs0[k];
    if (p != p0) read_batch(a.refs, p, p1, lane, 1, got);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) free += __popc(__ballot_sync(0xffffffffu, got[k] == 0));
  }
  if (lane == 0) {
    sm.warp_need[warp] = need;
    sm.warp_free[warp] = free;
  }
  __syncthreads();
  if (warp < 2) {  // exclusive sums over the CTA's warps; totals to every CTA
    int* mine = warp == 0 ? sm.warp_need : sm.warp_free;
    int* totals = warp == 0 ? sm.need : sm.free;
    int total;
    mine[lane] = sums_before(mine[lane], most, lane, &total);
    if (ctas == 1) {
      if (lane == 0) totals[0] = total;
    } else if (lane < ctas) {
      *cluster.map_shared_rank(totals + me, lane) = total;
    }
  }
  cluster.sync();
  int need_before = sm.warp_need[warp], free_before = sm.warp_free[warp];
  int total_need = 0, total_free = 0;
  for (int c = 0; c < ctas; ++c) {
    if (c < me) {
      need_before = sum_cut(need_before, sm.need[c], most);
      free_before += sm.free[c];
    }
    total_need = sum_cut(total_need, sm.need[c], most);
    total_free += sm.free[c];
  }
  if (total_need == 0 && !FORK) return;  // the same for all
  // The free pages by rank, as far as they are needed.
  const bool local = ctas == 1 && total_need <= kLocalList;
  int* list = local ? sm.list : x.list;
  for (int p = p0; p < p1 && free_before < total_need; p += 32 * kBatch) {
    int got[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) got[k] = refs0[k];
    if (p != p0) read_batch(a.refs, p, p1, lane, 1, got);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const unsigned hits = __ballot_sync(0xffffffffu, got[k] == 0);
      const int rank = free_before + __popc(hits & ((1u << lane) - 1));
      if (got[k] == 0 && rank < total_need) list[rank] = p + 32 * k + lane;
      free_before += __popc(hits);
    }
  }
  if (total_need > total_free && gw == 0 && lane == 0) raise_flag(a.status, WF_DEV_NO_PAGE);
  if (FORK && gw == 0 && lane == 0) *x.n_copies = min(total_need, total_free);
  if (local) {
    __syncthreads();
  } else {
    __threadfence();
    cluster.sync();
  }
  for (int u = u0; u < u1; ++u) {
    const int base = x.base[u];
    if (FORK && base < 0) continue;
    int rank = sum_cut(need_before, base, most);
    if (FORK) {
      const ForkUnit f = u == u0 ? fork0 : fork_unit(x, sm, u, false);
      const int32_t* from = a.table + static_cast<int64_t>(f.src) * a.table_pages;
      int32_t* to = a.table + static_cast<int64_t>(f.dst) * a.table_pages;
      // Behind the entries the child's are -1 already, as a rule.
      const int end = __any_sync(0xffffffffu, odd) ? a.table_pages : f.entries;
      for (int e0 = 0; e0 < end; e0 += 32 * kBatch) {
        int parents[kBatch], place[kBatch], fresh[kBatch];
        read_batch(from, e0, f.entries, lane, -1, parents);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const bool wants = parents[k] >= 0 && e0 + 32 * k + lane >= f.shared;
          const unsigned hits = __ballot_sync(0xffffffffu, wants);
          place[k] = rank + __popc(hits & ((1u << lane) - 1));
          fresh[k] = wants && place[k] < total_free ? list[place[k]] : -1;
          rank += __popc(hits);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int e = e0 + 32 * k + lane;
          if (e >= a.table_pages) continue;
          int page = -1;
          if (parents[k] >= 0) {
            const bool there = parents[k] < a.n_pages;
            if (!there) raise_flag(a.status, WF_DEV_BAD_INDEX);
            if (e < f.shared) {
              if (there) {
                page = parents[k];
                atomicAdd(a.refs + page, 1);
              }
            } else if (fresh[k] >= 0) {
              page = fresh[k];
              a.refs[page] = 1;
              x.copies[place[k]] = make_int4(there ? parents[k] : -1, page,
                                             min(a.page_size, f.len - e * a.page_size), 0);
            }
          }
          to[e] = page;
        }
      }
    } else {
      const ReserveUnit unit = u == u0 ? unit0 : reserve_unit<FROM>(x, u, false);
      int32_t* row = a.table + static_cast<int64_t>(u) * a.table_pages;
      for (int e0 = unit.first; e0 < unit.end; e0 += 32 * kBatch) {
        int got[kBatch], page[kBatch];
        read_batch(row, e0, unit.end, lane, 0, got);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const unsigned hits = __ballot_sync(0xffffffffu, got[k] < 0);
          const int r = rank + __popc(hits & ((1u << lane) - 1));
          page[k] = got[k] < 0 && r < total_free ? list[r] : -1;
          rank += __popc(hits);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          if (page[k] < 0) continue;
          row[e0 + 32 * k + lane] = page[k];
          a.refs[page[k]] = 1;
        }
      }
    }
  }
}

// Whole rows of pages: unit = (copy, pool, head), a warp each.
__global__ void __launch_bounds__(kThreads)
    copy_pages_kernel(const AllocArgs x, const PagePools pools, int row_chunks) {
  constexpr int kFly = 8;
  launch_dependents();
  wait_for_primary();
  const PagesArgs& a = x.p;
  const int lane = threadIdx.x & 31;
  const int per_copy = pools.n * a.kv_heads;
  const int64_t units = static_cast<int64_t>(*x.n_copies) * per_copy;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < units;
       u += step) {
    const int copy = static_cast<int>(u / per_copy);
    const int rest = static_cast<int>(u - static_cast<int64_t>(copy) * per_copy);
    const int pool = rest / a.kv_heads, head = rest - pool * a.kv_heads;
    const int4 c = x.copies[copy];
    if (c.x < 0) continue;
    uint4* base = static_cast<uint4*>(pools.at[pool]);
    const int64_t line = static_cast<int64_t>(a.page_size) * row_chunks;  // chunks of a head's rows
    const uint4* from = base + (static_cast<int64_t>(c.x) * a.kv_heads + head) * line;
    uint4* to = base + (static_cast<int64_t>(c.y) * a.kv_heads + head) * line;
    const int chunks = c.z * row_chunks;
    for (int i = lane; i < chunks; i += 32 * kFly) {
      uint4 v[kFly];
#pragma unroll
      for (int k = 0; k < kFly; ++k)
        if (i + 32 * k < chunks) v[k] = __ldcs(from + i + 32 * k);
#pragma unroll
      for (int k = 0; k < kFly; ++k)
        if (i + 32 * k < chunks) to[i + 32 * k] = v[k];
    }
  }
}

__global__ void __launch_bounds__(kThreads) release_kernel(const PagesArgs a, const int32_t* first,
                                                           const int32_t* end) {
  launch_dependents();
  wait_for_primary();
  for (int s = blockIdx.x; s < a.n_seqs; s += gridDim.x) {
    const int lo = min(max(ld(first + s), 0), max_len(a));
    const int hi = min(max(ld(end + s), 0), max_len(a));
    // Pages all of whose rows lie in [lo, hi).
    drop_entries(a, s, (lo + (a.page_size - 1)) / a.page_size, hi / a.page_size, threadIdx.x,
                 kThreads);
  }
}

// ---------------------------------------------------------------- kept rows
// Checks one sequence's list, resolves the rows that move and leaves in
// info[s] = (rows at the head that stay where they are, rows in all, new length
// or -1 when the sequence is left as it was).
constexpr int kPlanThreads = 1024, kPlanBatch = 4;
__global__ void __launch_bounds__(kPlanThreads) keep_plan_kernel(const KeepArgs x) {
  const PagesArgs& a = x.p;
  __shared__ int s_bad, s_shared, s_stay;
  const int threads = blockDim.x;
  launch_dependents();
  wait_for_primary();
  for (int s = blockIdx.x; s < a.n_seqs; s += gridDim.x) {
    __syncthreads();
    if (threadIdx.x == 0) s_bad = s_shared = 0;
    const int32_t* keep = x.keep + static_cast<int64_t>(s) * x.max_keep;
    const int32_t* row = a.table + static_cast<int64_t>(s) * a.table_pages;
    // The list's first rows come in beside its length.
    int from[kPlanBatch], prev[kPlanBatch];
    const auto read_rows = [&](int i0) {
#pragma unroll
      for (int k = 0; k < kPlanBatch; ++k) {
        const int i = i0 + k * threads;
        from[k] = i < x.max_keep ? ld(keep + i) : -1;
        prev[k] = i > 0 && i < x.max_keep ? ld(keep + i - 1) : -1;
      }
    };
    read_rows(threadIdx.x);
    const int len = ld(x.kv_len + s), start = ld(x.start + s);
    const int n = x.n_keep != nullptr ? ld(x.n_keep + s) : 0;
    const bool sound = len >= 0 && len <= max_len(a) && start >= 0 && start <= len && n >= 0 &&
                       n <= x.max_keep;
    const int count = sound ? n : 0;
    if (threadIdx.x == 0) s_stay = count;
    __syncthreads();
    bool bad = !sound, shared = false;
    for (int i0 = threadIdx.x; i0 < count; i0 += threads * kPlanBatch) {
      int page[kPlanBatch], to[kPlanBatch];
      if (i0 != threadIdx.x) read_rows(i0);
      // from = -1: a row that stays (so do all before it), or none, or one that
      // breaks the rules.  An ascending list's row i is start + i or behind it, so
      // that start + i lies in the table too.
#pragma unroll
      for (int k = 0; k < kPlanBatch; ++k) {
        const int i = i0 + k * threads;
        page[k] = to[k] = 0;
        if (i >= count) {
          from[k] = -1;
          continue;
        }
        if (from[k] <= prev[k] || from[k] < start || from[k] - start < i || from[k] >= len) {
          bad = true;
          from[k] = -1;
        } else if (from[k] - start == i) {
          from[k] = -1;
        } else {
          page[k] = row[from[k] / a.page_size];
          to[k] = row[(start + i) / a.page_size];
        }
      }
#pragma unroll
      for (int k = 0; k < kPlanBatch; ++k) {
        const int i = i0 + k * threads;
        if (from[k] < 0) continue;
        atomicMin(&s_stay, i);
        if (static_cast<unsigned>(page[k]) >= static_cast<unsigned>(a.n_pages) ||
            static_cast<unsigned>(to[k]) >= static_cast<unsigned>(a.n_pages))
          bad = true;
        else if (a.refs != nullptr && a.refs[to[k]] > 1)
          shared = true;
        x.lines[static_cast<int64_t>(s) * x.max_keep + i] =
            page[k] * a.page_size + (from[k] & (a.page_size - 1));
      }
    }
    if (bad) s_bad = 1;
    if (shared) s_shared = 1;
    __syncthreads();
    if (threadIdx.x == 0) {
      if (s_bad) raise_flag(a.status, WF_DEV_BAD_INDEX);
      if (s_shared) raise_flag(a.status, WF_DEV_SHARED_PAGE);
      const bool skip = s_bad || s_shared;
      x.info[s] = skip ? make_int4(0, 0, -1, 0) : make_int4(s_stay, count, start + count, start);
    }
  }
}

// Streams (sequence, pool, head, 128-byte piece of a row), each by GROUP
// threads, kRows of them a step's rows side by side, kFly steps' worth in
// flight twice.
constexpr int kPiece = 8;  // 16-byte chunks
template <int GROUP>
__global__ void __launch_bounds__(kThreads)
    move_rows_kernel(const KeepArgs x, const PagePools pools, int row_chunks, int page_shift) {
  constexpr int kFly = 4, kSide = GROUP / kPiece, kStep = kFly * kSide;
  const PagesArgs& a = x.p;
  launch_dependents();
  wait_for_primary();
  const int thread = GROUP == 32 ? threadIdx.x & 31 : threadIdx.x;
  const int pieces = row_chunks / kPiece, heads = a.kv_heads;
  const int per_seq = max(1, pools.n * heads * pieces);
  const int64_t streams = static_cast<int64_t>(a.n_seqs) * per_seq;
  const int groups = kThreads / GROUP;
  const auto meet = [] {
    if (GROUP == 32) __syncwarp(); else __syncthreads();
  };
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * groups + threadIdx.x / GROUP; w < streams;
       w += static_cast<int64_t>(gridDim.x) * groups) {
    const int s = static_cast<int>(w / per_seq);
    const int rest = static_cast<int>(w - static_cast<int64_t>(s) * per_seq);
    const int4 info = x.info[s];
    if (rest == 0 && info.z >= 0 && a.refs != nullptr)
      drop_entries(a, s, (info.z + a.page_size - 1) >> page_shift, a.table_pages, thread, GROUP);
    if (info.x >= info.y) continue;  // the same for the whole group
    const int piece = rest % pieces, head = rest / pieces % heads, pool = rest / pieces / heads;
    uint4* base = static_cast<uint4*>(pools.at[pool]) + piece * kPiece + thread % kPiece;
    const int32_t* lines = x.lines + static_cast<int64_t>(s) * x.max_keep;
    const int32_t* row = a.table + static_cast<int64_t>(s) * a.table_pages;
    // Chunk offset of a cache line (page * page_size + row) of this head.
    const auto place = [&](int page, int r) {
      return ((static_cast<int64_t>(page) * heads + head) * a.page_size + r) * row_chunks;
    };
    const int mask = a.page_size - 1;
    uint4 v[2][kFly];
    int next[kFly];
    const auto read_lines = [&](int i0) {
#pragma unroll
      for (int k = 0; k < kFly; ++k) {
        const int i = i0 + k * kSide + thread / kPiece;
        next[k] = i < info.y ? lines[i] : -1;
      }
    };
    const auto read_rows = [&](uint4* to) {
#pragma unroll
      for (int k = 0; k < kFly; ++k)
        if (next[k] >= 0) to[k] = base[place(next[k] >> page_shift, next[k] & mask)];
    };
    const auto write_rows = [&](const uint4* from, int i0) {
#pragma unroll
      for (int k = 0; k < kFly; ++k) {
        const int i = i0 + k * kSide + thread / kPiece, at = info.w + i;
        if (i < info.y) base[place(row[at >> page_shift], at & mask)] = from[k];
      }
    };
    int i = info.x;
    read_lines(i);
    read_rows(v[0]);
    read_lines(i + kStep);
    while (true) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        read_rows(v[b ^ 1]);
        read_lines(i + 2 * kStep);
        meet();  // every row of this step has been read
        write_rows(v[b], i);
        i += kStep;
        if (i >= info.y) break;
      }
      if (i >= info.y) break;
    }
  }
}

int row_chunks_of(const PagesArgs& a) { return a.head_dim * (a.dtype == WF_BF16 ? 2 : 4) / 16; }

unsigned grid_of(int64_t blocks) {
  return static_cast<unsigned>(
      std::max<int64_t>(1, std::min<int64_t>(blocks, 8 * device_sm_count())));
}

// A pool of many pages takes a cluster.
template <bool FORK, bool FROM>
cudaError_t launch_alloc(const AllocArgs& x, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(x.p.n_pages <= kOneCta ? 1 : kAllocCluster);
  cfg.blockDim = dim3(kAllocThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {cfg.gridDim.x, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = cfg.gridDim.x == 1 ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, alloc_kernel<FORK, FROM>, x);
}

}  // namespace

cudaError_t launch_reserve(const AllocArgs& x, cudaStream_t stream) {
  return x.from != nullptr ? launch_alloc<false, true>(x, stream)
                           : launch_alloc<false, false>(x, stream);
}

cudaError_t launch_fork(const AllocArgs& x, const PagePools& pools, cudaStream_t stream) {
  const cudaError_t e = launch_alloc<true, false>(x, stream);
  if (e != cudaSuccess) return e;
  const int64_t most =
      std::min<int64_t>(x.p.n_pages, static_cast<int64_t>(x.units) * x.p.table_pages);
  return launch_early(copy_pages_kernel, dim3(grid_of(most * pools.n * x.p.kv_heads / kWarps + 1)),
                      kThreads, 0, stream, x, pools, row_chunks_of(x.p));
}

cudaError_t launch_release(const PagesArgs& a, const int32_t* first, const int32_t* end,
                           cudaStream_t stream) {
  return launch_early(release_kernel, dim3(grid_of(a.n_seqs)), kThreads, 0, stream, a, first, end);
}

cudaError_t launch_keep(const KeepArgs& x, const PagePools& pools, cudaStream_t stream) {
  const cudaError_t e =
      launch_early(keep_plan_kernel, dim3(grid_of(x.p.n_seqs)),
                   x.max_keep > kThreads ? kPlanThreads : kThreads, 0, stream, x);
  if (e != cudaSuccess) return e;
  const int chunks = row_chunks_of(x.p);
  int shift = 0;
  while ((1 << shift) < x.p.page_size) ++shift;
  // A warp a stream where lists are short (an accepted path), else a CTA.
  const int64_t streams = static_cast<int64_t>(x.p.n_seqs) *
                          std::max(1, pools.n * x.p.kv_heads * (chunks / kPiece));
  const bool warps = x.max_keep <= 32;
  const dim3 grid(grid_of(warps ? (streams + kWarps - 1) / kWarps : streams));
  return warps ? launch_early(move_rows_kernel<32>, grid, kThreads, 0, stream, x, pools, chunks,
                              shift)
               : launch_early(move_rows_kernel<kThreads>, grid, kThreads, 0, stream, x, pools,
                              chunks, shift);
}

}  // namespace wf
