// Shared pieces of the dense attention kernels (paged cache and packed
// prompts): the sizes and options handed to the launchers, the scores'
// transformation and mask, and the division of the paged cache's key tiles
// over a persistent grid.
//
// Scores.  For query position p and key j of one sequence
//   z = scale q·k;  z <- c tanh(z / c) (c > 0);  z <- z - slope_h |p - j|
// and key j counts when j < len and (not causal, or j <= p, or j < prefix).
// Kernels keep z in the log2 domain (times log2 e) in fp32; O = Σ 2^(z-m) v /
// Σ 2^(z-m).  A row without a visible key yields O = 0, lse = -inf.
#pragma once

#include <cmath>

#include "wf_common.cuh"
#include "wf_internal.h"

namespace wf {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Options of one launch, scores already in the log2 domain.
struct ScoreOpts {
  float scale;            // scale * log2 e without a cap, else scale / cap
  float cap;              // cap * log2 e, or 0
  float bend_max;         // largest |scale s| the cap's polynomial may take (-1: none)
  const int32_t* prefix;  // nullable
  const float* slopes;    // nullable
  int causal;
};

// tanh(x) / x as a polynomial of x^2 for |x| <= 1/2: Chebyshev interpolation
// on [0, 1/4], error of tanh below 2^-22 relative with the fp32 roundings.
constexpr float kBend[5] = {1.f, -0.333330721f, 0.133248284f, -0.0529892407f, 0.0171413198f};

// tanh by that polynomial for small arguments, else 1 - 2 / (1 + e^(2x)) with
// the hardware 2^x and reciprocal approximations (absolute error below 2^-21):
// relative error below 2^-20 either way, whatever the cap.
__device__ __forceinline__ float tanh_exp2(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + fast_exp2(x * (2.f * kLog2e))));
  const float u = x * x;
  const float q =
      fmaf(fmaf(fmaf(fmaf(kBend[4], u, kBend[3]), u, kBend[2]), u, kBend[1]), u, kBend[0]);
  return fabsf(x) <= 0.5f ? x * q : fmaf(-2.f, r, 1.f);
}

// Reciprocal of a softmax sum and the row's lse from its log2-domain maximum
// and sum.  The sum is 0 only for a row without a visible key (the maximum
// itself contributes 1); a NaN among the visible scores stays NaN.
__device__ __forceinline__ float inv_or_zero(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float row_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Keys visible to some row of [first, last] query positions of a sequence:
// the exclusive end of the key range the rows need.
__device__ __forceinline__ int visible_end(int len, int last_pos, int causal, int prefix) {
  return causal ? min(len, max(last_pos + 1, prefix)) : len;
}

inline ScoreOpts score_opts(float scale, float softcap, int causal, const int32_t* prefix,
                            const float* slopes) {
  ScoreOpts o;
  o.cap = softcap > 0.f ? softcap * kLog2e : 0.f;
  o.scale = softcap > 0.f ? scale / softcap : scale * kLog2e;
  // The polynomial's coefficients are cap scale^1, ^3 .. ^9 times numbers of
  // 0.017 to 1: all are normal floats where the last one is well inside.
  const double last = static_cast<double>(o.cap) * std::pow(static_cast<double>(o.scale), 9.0);
  o.bend_max = last > 1e-30 && last < 1e30 ? 0.5f : -1.f;
  o.causal = causal;
  o.prefix = prefix;
  o.slopes = slopes;
  return o;
}

__device__ __forceinline__ void store4(float* dst, const float* f) {
  *reinterpret_cast<float4*>(dst) = make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* dst, const float* f) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), c = __floats2bfloat162_rn(f[2], f[3]);
  *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                              *reinterpret_cast<const uint32_t*>(&c));
}

// What the bounded waits of a CTA share (shared memory).
struct WaitState {
  int abort;       // a wait of this CTA has given up
  uint32_t polls;  // the limit of each
  __device__ __forceinline__ void init(uint32_t limit) {
    abort = 0;
    polls = limit;
  }
};

// A bounded wait on an mbarrier phase by a whole converged warp, which also
// ends when another warp of the CTA has given up; true when the phase has
// completed.  The first tries stand alone, outside any loop: a try
// sleeps until the phase completes or its time limit, so it usually
// suffices, and a wait that is over already costs 70 cycles this way against
// 220 in the loop (measured in the packed-prompt kernel, whose products wait
// four times a key tile).  `nap`: nanoseconds between the later polls, for
// warps with time to spare.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, WaitState& w,
                                          int32_t* status, uint32_t nap = 0) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const uint32_t polls = w.polls;
  for (uint32_t i = 0; i < polls; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (nap != 0) __nanosleep(nap);
    if ((i & 255) == 255 &&
        __any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&w.abort) != 0))
      return false;
  }
  raise_flag(status, WF_DEV_WAIT_TIMEOUT);
  *reinterpret_cast<volatile int*>(&w.abort) = 1;
  return false;
}

// Programmatic dependent launch: the next kernel of the stream (launched with
// that attribute) may start its prologue; it waits for this one's results.
__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_primary() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ---------------------------------------------------------------- paged work list
// The key tiles of every unit (sequence, key-value head, row block) in one
// line: sequence by sequence, unit by unit, tile by tile.  CTA c of C takes
// the tiles [W c / C, W (c + 1) / C): even work whatever the lengths, and a
// unit's tiles lie with consecutive CTAs.  A CTA holding a whole unit writes
// the output; otherwise each CTA leaves one partial (m, l, O) per unit, in
// its slot 2c (the unit its range starts inside of) or 2c + 1 (the unit its
// range ends inside of), and the join kernel merges consecutive CTAs' slots
// in order (fixed order: bit-identical from run to run).
struct WorkShape {
  int n_seqs;
  int units_per_seq;  // kv_heads * row blocks
  int tile;           // keys per tile
  int max_len;        // table_pages * page_size
};

// Tiles of one sequence: its length clamped into the table (a longer one is
// flagged by the caller).
__device__ __forceinline__ int seq_len_clamped(const int32_t* lens, int s, int max_len) {
  return min(max(__ldg(lens + s), 0), max_len);
}

__device__ __forceinline__ int seq_tiles(const WorkShape& w, const int32_t* lens, int s) {
  return (seq_len_clamped(lens, s, w.max_len) + w.tile - 1) / w.tile;
}

// Tiles of the whole call.  Whole warp.
__device__ __forceinline__ int64_t work_total(const WorkShape& w, const int32_t* lens) {
  int n = 0;  // fits: the host bounds n_seqs times the longest sequence's tiles
  for (int s = threadIdx.x & 31; s < w.n_seqs; s += 32) n += seq_tiles(w, lens, s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return static_cast<int64_t>(n) * w.units_per_seq;
}

// First tiles of the CTAs' ranges: CTA c of n starts at c q + c r / n with
// total = q n + r.  With fewer tiles than CTAs, one tile each for the first
// ones: no CTA between two that share a unit is ever idle.
struct WorkSplit {
  int64_t total, q;
  uint32_t r, n;
  __device__ __forceinline__ WorkSplit(int64_t total_, int n_)
      : total(total_), n(static_cast<uint32_t>(n_)) {
    if (total < n) {
      q = 1;
      r = 0;
    } else if (total >> 32 == 0) {  // 32-bit division where it does
      q = static_cast<uint32_t>(total) / n;
      r = static_cast<uint32_t>(total) - static_cast<uint32_t>(q) * n;
    } else {
      q = total / n;
      r = static_cast<uint32_t>(total - q * n);
    }
  }
  __device__ __forceinline__ int64_t begin(int c) const {
    return min(total, c * q + static_cast<uint32_t>(c) * r / n);
  }
  // The CTA whose range holds tile t: the largest c with begin(c) <= t, that
  // is floor(c total / n) <= t, c < (t + 1) n / total.
  __device__ __forceinline__ int owner(int64_t t) const {
    if (total < n) return static_cast<int>(t);
    const uint64_t x = static_cast<uint64_t>(t + 1) * n + static_cast<uint64_t>(total) - 1;
    return static_cast<int>(x >> 32 == 0
                                ? static_cast<uint32_t>(x) / static_cast<uint32_t>(total)
                                : x / static_cast<uint64_t>(total)) - 1;
  }
};

// A unit: its sequence and length, its index within the sequence, its tiles
// and the first of them.
struct WorkUnit {
  int seq, len, unit, tiles;
  int64_t begin;
};
// The unit that holds tile `at` (0 <= at < total).  Whole warp, 32 sequences
// a step.
__device__ __forceinline__ WorkUnit find_unit(const WorkShape& w, const int32_t* lens,
                                              int64_t at) {
  const int lane = threadIdx.x & 31;
  int base = 0;
  WorkUnit u = {0, 0, 0, 1, 0};
  for (int s0 = 0; s0 < w.n_seqs; s0 += 32) {
    const int len = s0 + lane < w.n_seqs ? seq_len_clamped(lens, s0 + lane, w.max_len) : 0;
    const int t = (len + w.tile - 1) / w.tile;
    const int incl = warp_incl_scan(t);
    const unsigned hit = __ballot_sync(
        0xffffffffu, static_cast<int64_t>(base + incl) * w.units_per_seq > at);
    if (hit != 0) {
      const int src = __ffs(hit) - 1;
      const int64_t first = static_cast<int64_t>(base + __shfl_sync(0xffffffffu, incl - t, src)) *
                            w.units_per_seq;
      u.seq = s0 + src;
      u.len = __shfl_sync(0xffffffffu, len, src);
      u.tiles = __shfl_sync(0xffffffffu, t, src);
      const int64_t off = at - first;  // below units_per_seq tiles
      u.unit = off >> 32 == 0
                   ? static_cast<int>(static_cast<uint32_t>(off) / static_cast<uint32_t>(u.tiles))
                   : static_cast<int>(off / u.tiles);
      u.begin = first + static_cast<int64_t>(u.unit) * u.tiles;
      return u;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return u;
}
// The unit after u (there is one: the caller stays below the total).  Whole
// warp, which looks at 32 sequences a step for one with keys where the next one
// is idle.
__device__ __forceinline__ void next_unit(const WorkShape& w, const int32_t* lens, WorkUnit& u) {
  u.begin += u.tiles;
  if (++u.unit < w.units_per_seq) return;
  u.unit = 0;
  const int lane = threadIdx.x & 31;
  ++u.seq;
  u.len = u.seq < w.n_seqs ? seq_len_clamped(lens, u.seq, w.max_len) : 0;
  for (int s0 = u.seq + 1; u.len == 0 && s0 < w.n_seqs; s0 += 32) {
    const int len = s0 + lane < w.n_seqs ? seq_len_clamped(lens, s0 + lane, w.max_len) : 0;
    const unsigned live = __ballot_sync(0xffffffffu, len > 0);
    if (live == 0) continue;
    u.seq = s0 + __ffs(live) - 1;
    u.len = __shfl_sync(0xffffffffu, len, __ffs(live) - 1);
  }
  u.tiles = (u.len + w.tile - 1) / w.tile;
}

// Rows of a sequence without keys: O = 0, lse = -inf.  CTA c of n, threads
// thread, thread + threads, ...; flags lengths outside the table.
template <typename T>
__device__ __forceinline__ void idle_sequences(const PagedArgs& a, int max_len, int c, int n,
                                               int thread, int threads) {
  for (int s = c; s < a.n_seqs; s += n) {
    const int len = __ldg(a.kv_len + s);
    if (thread == 0 && (len < 0 || len > max_len)) raise_flag(a.status, WF_DEV_BAD_INDEX);
    if (len > 0) continue;
    const int rows = a.n_new * a.q_heads;
    uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(a.o) +
                                        static_cast<int64_t>(s) * rows * a.head_dim);
    const int chunks = rows * (a.head_dim / Elem<T>::kPer16B);
    for (int e = thread; e < chunks; e += threads) o[e] = make_uint4(0u, 0u, 0u, 0u);
    if (a.lse != nullptr)
      for (int e = thread; e < rows; e += threads)
        a.lse[static_cast<int64_t>(s) * rows + e] = -INFINITY;
  }
}

// Kernel parameters of the paged attention.
struct PagedParams {
  PagedArgs a;
  WorkShape w;
  ScoreOpts o;
  int row_blocks;
};
inline PagedParams paged_params(const PagedArgs& a, const PagedPlan& plan) {
  PagedParams p;
  p.a = a;
  p.row_blocks = (a.q_heads / a.kv_heads * a.n_new + plan.row_block - 1) / plan.row_block;
  p.w.n_seqs = a.n_seqs;
  p.w.units_per_seq = a.kv_heads * p.row_blocks;
  p.w.tile = kPagedTile;
  p.w.max_len = a.table_pages * a.page_size;
  p.o = score_opts(a.scale, a.softcap, a.causal, a.prefix, a.slopes);
  return p;
}

// ---------------------------------------------------------------- packed row blocks
// Row blocks of packed sequences: `rows` rows of one key-value head a block
// (n_q g rows in a sequence).  doc_blocks() blocks cover any split of the rows
// into sequences; a padded batch (many empty sequences) has far fewer, so that
// grids are capped and their blocks then share out what doc_total() counts.
// find_doc_block maps a block index to its sequence (whole warp; false: past
// the last block).  Offsets are clamped into the arrays, and a bad one is
// flagged.
inline int64_t doc_blocks(int64_t rows_q, int n_docs, int rows, int g) {
  return rows_q * g / rows + n_docs;
}
struct DocBlock {
  int doc, block;   // sequence, row block within it
  int n_q, n_k;     // its rows and keys
  int64_t q0, k0;   // its first row and key
};
__device__ __forceinline__ int doc_span(const int32_t* cu, int i, int rows, int* first) {
  const int a = min(max(__ldg(cu + i), 0), rows), b = min(max(__ldg(cu + i + 1), 0), rows);
  *first = a;
  return max(b - a, 0);
}
// Row blocks of all sequences.  Whole warp.
__device__ __forceinline__ int64_t doc_total(const PrefillArgs& a, int rows, int g) {
  int64_t n = 0;
#pragma unroll 4
  for (int d = threadIdx.x & 31; d < a.n_docs; d += 32) {
    int first;
    n += (static_cast<int64_t>(doc_span(a.cu_q, d, a.rows_q, &first)) * g + rows - 1) / rows;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n;
}
// Where the last search ended: its 32 sequences and the blocks before them
// (behind the last sequence: all).
struct DocCursor {
  int d0;
  int64_t base;
};
__device__ __forceinline__ bool find_doc_block(const PrefillArgs& a, int64_t at, int rows, int g,
                                               DocCursor& cursor, DocBlock* out) {
  const int lane = threadIdx.x & 31;
  // The warp scans the sequences, 32 at a time.
  if (at < cursor.base) cursor = {0, 0};
  int64_t base = cursor.base;
  for (int d0 = cursor.d0; d0 < a.n_docs; d0 += 32) {
    int first = 0, n = 0;
    if (d0 + lane < a.n_docs) n = doc_span(a.cu_q, d0 + lane, a.rows_q, &first);
    const int blocks = static_cast<int>((static_cast<int64_t>(n) * g + rows - 1) / rows);
    const int incl = warp_incl_scan(blocks);
    const unsigned hit = __ballot_sync(0xffffffffu, base + incl > at);
    if (hit != 0) {
      const int src = __ffs(hit) - 1;
      out->doc = d0 + src;
      out->block = static_cast<int>(at - base) - __shfl_sync(0xffffffffu, incl - blocks, src);
      out->q0 = __shfl_sync(0xffffffffu, first, src);
      out->n_q = __shfl_sync(0xffffffffu, n, src);
      int k0 = 0;
      out->n_k = doc_span(a.cu_k, out->doc, a.rows_k, &k0);
      out->k0 = k0;
      cursor = {d0, base};
      return true;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  cursor = {a.n_docs, base};
  return false;
}

// Flags offsets that are not ascending within [0, rows] (one block checks).
__device__ __forceinline__ void check_offsets(const int32_t* cu, int n, int rows, int32_t* status,
                                              int thread, int threads) {
  for (int i = thread; i < n; i += threads) {
    const int a = __ldg(cu + i), b = __ldg(cu + i + 1);
    if (a < 0 || b < a || b > rows) raise_flag(status, WF_DEV_BAD_INDEX);
  }
}

}  // namespace wf
