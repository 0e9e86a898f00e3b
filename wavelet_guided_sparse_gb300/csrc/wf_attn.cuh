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

#include "wf_common.cuh"
#include "wf_internal.h"

namespace wf {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Options of one launch, scores already in the log2 domain.
struct ScoreOpts {
  float scale;            // scale * log2 e without a cap, else scale / cap
  float cap;              // cap * log2 e, or 0
  const int32_t* prefix;  // nullable
  const float* slopes;    // nullable
  int causal;
};

// tanh(x) = 1 - 2 / (1 + e^(2x)), with the hardware 2^x and reciprocal
// approximations: absolute error below 2^-21, which moves a score by less
// than cap * 2^-21 (the same order as the fp32 rounding of q·k).
__device__ __forceinline__ float tanh_exp2(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + fast_exp2(x * (2.f * kLog2e))));
  return fmaf(-2.f, r, 1.f);
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

// Exclusive prefix sums of the sequences' tile counts into pre[0..n_seqs]
// (shared memory).  Whole block; contains __syncthreads.
__device__ __forceinline__ void work_prefix(const WorkShape& w, const int32_t* lens, int* pre,
                                            int* scratch) {
  int base = 0;
  for (int s0 = 0; s0 < w.n_seqs; s0 += kThreads) {
    const int s = s0 + threadIdx.x;
    const int t =
        s < w.n_seqs ? (seq_len_clamped(lens, s, w.max_len) + w.tile - 1) / w.tile : 0;
    int total;
    const int e = block_excl_scan(t, scratch, &total);
    if (s < w.n_seqs) pre[s] = base + e;
    base += total;
  }
  if (threadIdx.x == 0) pre[w.n_seqs] = base;
  __syncthreads();
}

// First tile of CTA c of n.  With fewer tiles than CTAs, one tile each for
// the first ones: no CTA between two that share a unit is ever idle.
__device__ __forceinline__ int64_t work_bound(int64_t total, int c, int n) {
  return total < n ? min(static_cast<int64_t>(c), total) : total * c / n;
}

// The unit that holds tile `at` (0 <= at < total): its sequence, its index
// within the sequence, its first tile and its tile count.
struct WorkUnit {
  int seq, unit, tiles;
  int64_t begin;
};
__device__ __forceinline__ WorkUnit find_unit(const WorkShape& w, const int* pre, int64_t at) {
  int lo = 0, hi = w.n_seqs;  // last s with pre[s] * units <= at
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (static_cast<int64_t>(pre[mid]) * w.units_per_seq <= at) lo = mid; else hi = mid;
  }
  // Sequences without tiles share their start with the next one: the last
  // with pre[s] * units <= at has tiles, because `at` is below its end.
  WorkUnit u;
  u.seq = lo;
  u.tiles = pre[lo + 1] - pre[lo];
  const int64_t off = at - static_cast<int64_t>(pre[lo]) * w.units_per_seq;
  u.unit = static_cast<int>(off / u.tiles);
  u.begin = static_cast<int64_t>(pre[lo]) * w.units_per_seq +
            static_cast<int64_t>(u.unit) * u.tiles;
  return u;
}

// ---------------------------------------------------------------- packed row blocks
// Row blocks of packed sequences: `rows` rows of one key-value head a block
// (n_q g rows in a sequence).  A grid of doc_blocks() blocks covers any split
// of the rows into sequences; find_doc_block maps a block index to its
// sequence (whole block; false: past the last block).  Offsets are clamped
// into the arrays, and a bad one is flagged.
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
__device__ __forceinline__ bool find_doc_block(const PrefillArgs& a, int64_t at, int rows, int g,
                                               DocBlock* out) {
  const int lane = threadIdx.x & 31;
  // Every warp scans the sequences, 32 at a time.
  int64_t base = 0;
  for (int d0 = 0; d0 < a.n_docs; d0 += 32) {
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
      return true;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

// Flags offsets that are not ascending within [0, rows] (one block checks).
__device__ __forceinline__ void check_offsets(const int32_t* cu, int n, int rows,
                                              int32_t* status) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int a = __ldg(cu + i), b = __ldg(cu + i + 1);
    if (a < 0 || b < a || b > rows) raise_flag(status, WF_DEV_BAD_INDEX);
  }
}

inline ScoreOpts score_opts(float scale, float softcap, int causal, const int32_t* prefix,
                            const float* slopes) {
  ScoreOpts o;
  o.cap = softcap > 0.f ? softcap * kLog2e : 0.f;
  o.scale = softcap > 0.f ? scale / softcap : scale * kLog2e;
  o.causal = causal;
  o.prefix = prefix;
  o.slopes = slopes;
  return o;
}

}  // namespace wf
