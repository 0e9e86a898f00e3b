// Drafted trees and sliding windows over a paged cache on the fifth-generation
// tensor cores (bf16): the split kernel where a sequence's g n_new query rows would
// make the paged mma.sync kernel (wf_paged_kernel.cuh) read its cache once for
// every 64 of them, and wherever its warps take turns in adding up.
//
// A unit is a (sequence, key-value head, row block); a row is (node or new token,
// query head), node-major, so that a tile of 128 rows holds 128 / g nodes with all
// their heads (one tensor copy; fewer rows where g does not divide 128).  The
// 128-key tiles of all units form the line of wf_attn.cuh, divided evenly over a
// persistent grid; parts of split units are joined by the paged join kernel.
//
// Two softmax groups of 128 threads, one thread a row, keep the tensor cores
// busy in turn, as in the packed-prompt kernel (wf_prefill.cu):
//   PAIR (more than one tile of rows): two row tiles over the same keys; per key
//         tile  PV_0 QK_0' PV_1 QK_1'  (' the next key tile);
//   else: one row tile, the groups take alternate key tiles, each with its own
//         maximum, sum and output; tensor memory holds both outputs in the same
//         lanes, so that at a unit's end each group adds up half of the columns.
// Products wait for keys ahead by one (PAIR) or two key tiles: K_0 .. K_{L-1},
// then V_i and K_{i+L} for i = 0, 1, ...  Warp 0 issues every product, warp 1
// the tensor copies of queries and keys, warp 2 those of values (whole pages or
// 128-row parts of them), warp 3 sees to idle sequences.  Keys run from a part's last
// tile to its first (the line of a window's key tiles has a gap behind the first
// tokens), so that the drafted rows, a tree's only ones with a mask, come first.
// Weights, maximum and roundings as in wf_prefill.cu: a weight meets one rounding to
// bf16, also with 5 to 16 rows, where the mma.sync kernel takes it in two parts
// (relative error against 64 bits 0.0020 to 0.0023 in place of 0.0017, the output's
// own rounding; that kernel needs 24.8 us where this one takes 18.9, see kFewRows).
//
// Rows behind a sequence's end and rows of bad pages get weights of exactly 0,
// and their value rows, up to the product's end, are cleared in shared memory.
// Query rows without a node compute something and are written as O = 0.
//
// Measured (32 query heads, 8 of keys, d = 128; bound by HBM, whose share is of one
// read of the cache): trees of 26 nodes over 16 sequences of 1000 to 16384 keys 91
// us, 71 %; of 64 nodes over four of 32768 keys 111 us, 72 %, with capped scores 161,
// with cap and bias 200 (the scores' mapping); 26 nodes over one of 131072 keys 95
// us, 83 %.  What is missing: 6 us to the first scores (lengths, tables and queries are
// read behind the last kernel's end), 1.5 us an output (a CTA's
// units follow one another), 6 us of join, and CTAs that end 5 us apart.  A softmax
// group takes about 2900 cycles a key tile of 128 rows, as long as HBM needs for its
// copy: with 128 rows two groups on alternate tiles leave room for the waits between
// the roles, with 256 they are the whole of it.
#pragma once

#include <algorithm>

#include "wf_attn_umma.cuh"
#include "wf_paged_kernel.cuh"
#include "wf_tensormap.h"

namespace wf {

namespace {

constexpr int kUmmaThreads = 384;
constexpr int kUmmaIssueRegs = 104, kUmmaSoftmaxRegs = 200;
static_assert(8 * kUmmaSoftmaxRegs + 4 * kUmmaIssueRegs <= 12 * 168, "beyond the launch's registers");

template <int D, bool PAIR>
struct UmmaShape {
  static constexpr int kTileBytes = kTileRows * D * 2;
  static constexpr int kQueryTiles = PAIR ? 2 : 1;
  static constexpr int kStages = D == 64 ? 8 : 5;
  // Alternate key tiles: (m, l) by unit parity, group and row.
  static constexpr size_t kSumBytes = PAIR ? 0 : 2 * 2 * kTileRows * 2 * sizeof(float);
  static constexpr size_t kSmem =
      1024 + (kQueryTiles + kStages) * static_cast<size_t>(kTileBytes) + kSumBytes;
};

struct UmmaParams {
  CUtensorMap tq, tk, tv;
  PagedParams p;
  int box_rows, page_shift;
  int tile_nodes, tile_rows;  // nodes and rows (nodes * g) of a query tile
  uint32_t inject_polls;      // fault injection (tests): see the kernel's start
};

struct UmmaBarriers {
  uint64_t full[8];            // ring stages
  uint64_t done[8];            // steps whose stages are free again
  uint64_t q, q_empty;         // query tiles in shared memory
  uint64_t s[2], p[2];         // scores ready; weights ready
  uint64_t o[2], o_empty[2];   // output finished; read
  uint64_t drain;
  int valid[8];                // of a key tile, by its number: one bit a box
  uint32_t issued[2][8];       // last fill of each stage by the copying warps, plus 1
  uint32_t tmem;
  WaitState wait;
};

__device__ __forceinline__ void tma_load_4d(void* dst, const void* tmap, int x, int y, int z, int w,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// The part of a unit that a CTA holds: key tiles [j0, j1), none where only the
// pad behind a unit's tiles lies in its range; `next`: where the next unit's begins.
struct UnitPart {
  int j0, j1;
  bool all;
  int64_t next;
};
__device__ __forceinline__ UnitPart unit_part(const WorkShape& w, const WorkUnit& u, int64_t at,
                                              int64_t w1) {
  UnitPart x;
  const int tiles = u.tiles - w.pad;
  x.next = min(w1, u.begin + u.tiles);
  x.j0 = static_cast<int>(at - u.begin);
  x.j1 = max(x.j0, min(static_cast<int>(x.next - u.begin), tiles));
  x.all = x.j0 == 0 && x.j1 == tiles;
  return x;
}

// Keys from the first of tile j of the line on that count: up to the sequence's
// end, or the first tokens'.
template <int MASK>
__device__ __forceinline__ int tile_keys(const WorkShape& w, const Span& x, int len, int j) {
  if (MASK == kMaskWindow && x.gap > 0 && j < x.first) return w.sinks - j * kTileRows;
  return len - x.place(j) * kTileRows;
}

// Bits of an ancestor mask for the 32 keys from `rel` nodes behind (before, if
// negative) the first drafted row on; rows before it are seen by all.
__device__ __forceinline__ uint32_t tree_bits(uint64_t up, int rel) {
  if (rel >= 0) return rel < 64 ? static_cast<uint32_t>(up >> rel) : 0u;
  return low_bits(-rel) | (rel > -32 ? static_cast<uint32_t>(up << -rel) : 0u);
}
// Bits of the 32 keys from row c of a key tile on that lie in boxes with a page.
__device__ __forceinline__ uint32_t box_bits(int valid, int c, int box_shift) {
  uint32_t bits = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b)
    bits |= (valid >> ((c + 8 * b) >> box_shift)) & 1 ? 0xffu << (8 * b) : 0u;
  return bits;
}

template <int D, bool PAIR, int MASK, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kUmmaThreads, 1)
    paged_umma_kernel(const __grid_constant__ UmmaParams tp) {
  using Shape = UmmaShape<D, PAIR>;
  constexpr int kStages = Shape::kStages, kTileBytes = Shape::kTileBytes;
  constexpr int KB = D / 64, kAhead = PAIR ? 1 : 2;
  constexpr int kBlock = kTileRows * 128;  // bytes of a 64-column block
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) UmmaBarriers bars;
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  unsigned char* ring = smem + Shape::kQueryTiles * kTileBytes;
  const PagedParams& p = tp.p;
  const PagedArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = a.q_heads / a.kv_heads;

  // Fault injection (tests of the bounded waits): the first CTA's first key tile
  // is never issued, and its waits give up after inject_polls polls.
  const bool inject = tp.inject_polls != 0 && blockIdx.x == 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 8; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.done[i], 1);
    }
    mbar_init(&bars.q, 1);
    mbar_init(&bars.q_empty, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars.s[t], 1);
      mbar_init(&bars.p[t], 128);
      mbar_init(&bars.o[t], 1);
      mbar_init(&bars.o_empty[t], PAIR ? 128 : 256);
    }
    mbar_init(&bars.drain, 1);
    bars.wait.init(inject ? tp.inject_polls : kWaitPolls);
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(&bars.tmem, 512);
  if (warp == 1 && lane == 0) {
    prefetch_tensormap(&tp.tq);
    prefetch_tensormap(&tp.tk);
    prefetch_tensormap(&tp.tv);
  }
  wait_for_primary();
  const WorkSplit split(work_total<MASK>(p.w, a.kv_len), gridDim.x);
  const int64_t w0 = split.begin(blockIdx.x), w1 = split.begin(blockIdx.x + 1);
  WorkUnit u = find_unit<MASK>(p.w, a.kv_len, w0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  launch_dependents();
  const uint32_t tmem = bars.tmem;
  const uint32_t tS[2] = {tmem, tmem + 128};
  const uint32_t tO[2] = {tmem + 256, tmem + 256 + D};
  const int RT = PAIR ? 2 * tp.tile_rows : kTileRows;  // rows of a row block
  // Row tiles of the unit's row block that have rows.
  const auto tiles_with_rows = [&](const WorkUnit& x) {
    const int row0 = (x.unit % p.row_blocks) * RT;
    return PAIR && g * a.n_new - row0 > tp.tile_rows ? 2 : 1;
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kUmmaIssueRegs));
    const bool leader = elect_one();
    if (warp == 3) {
      idle_sequences<__nv_bfloat16, MASK>(a, p.w, blockIdx.x, gridDim.x, lane, 32);
    } else if (warp > 0) {
      // ---- copies: lane = (box, column block) of a stage.  Both warps walk all
      // fills; warp 1 issues queries and keys, warp 2 values.
      const bool keys = warp == 1;
      const int boxes = kTileRows / tp.box_rows;
      const int box = lane / KB, kb = lane % KB;
      const uint32_t box_bytes = static_cast<uint32_t>(tp.box_rows) * 128;
      const unsigned every = __ballot_sync(0xffffffffu, box < boxes);
      bool ok = true;
      uint32_t fills = 0, steps = 0, tiles = 0, units = 0;
      uint32_t step_of[kStages] = {};  // the step that frees each stage
      uint32_t mine[kStages] = {};     // this warp's last fill of each, plus 1
      int st = 0;
      Span span = span_of<MASK>(p.w, u.len);
      // First row of this lane's box of tile j of the line, and its page-table entry
      // (-1: nothing to copy).
      const auto box_key = [&](int j) { return span.place(j) * kTileRows + box * tp.box_rows; };
      const auto entry = [&](int j) {
        const int key = box_key(j);
        return box < boxes && box_needed<MASK>(p.w, span, u.len, key, tp.box_rows)
                   ? load_input<kReadOrdered>(a.table +
                                              static_cast<int64_t>(u.seq) * a.table_pages +
                                              (key >> tp.page_shift))
                   : -1;
      };
      const auto fill = [&](bool key_fill, int j, int page, int kvh, uint32_t step) {
        if (key_fill == keys) {
          if (fills >= kStages) {
            uint32_t r = 0;
#pragma unroll
            for (int i = 0; i < kStages; ++i) r = i == st ? step_of[i] : r;
            ok = ok && warp_wait(&bars.done[r & 7], (r >> 3) & 1, bars.wait, a.status);
          }
          if (!ok) return;
          const int key = box_key(j);
          const unsigned live = __ballot_sync(
              0xffffffffu, static_cast<unsigned>(page) < static_cast<unsigned>(a.n_pages));
          if (!((live >> lane) & 1) && box < boxes &&
              box_needed<MASK>(p.w, span, u.len, key, tp.box_rows))
            raise_flag(a.status, WF_DEV_BAD_INDEX);
          const bool issue = !(inject && fills == 0);
          if (lane == 0 && issue) {
            if (keys) {
              int valid = (1 << boxes) - 1;
              if (live != every)
                for (int b = 0; b < boxes; ++b)
                  if (!((live >> (b * KB)) & 1)) valid &= ~(1 << b);
              bars.valid[tiles & 7] = valid;
            }
            mbar_arrive_expect_tx(&bars.full[st], __popc(live) * box_bytes);
          }
          __syncwarp();
          if (issue && ((live >> lane) & 1))
            tma_load_2d(ring + st * kTileBytes + kb * kBlock + box * box_bytes,
                        keys ? &tp.tk : &tp.tv, kb * 64,
                        (page * a.kv_heads + kvh) * a.page_size + (key & (a.page_size - 1)),
                        &bars.full[st]);
#pragma unroll
          for (int i = 0; i < kStages; ++i)
            if (i == st && issue) mine[i] = fills + 1;
        }
#pragma unroll
        for (int i = 0; i < kStages; ++i)
          if (i == st) step_of[i] = step;
        tiles += key_fill;
        ++fills;
        if (++st == kStages) st = 0;
      };
      const auto to_next = [&]() {
        next_unit<MASK>(p.w, a.kv_len, u);
        span = span_of<MASK>(p.w, u.len);
      };
      for (int64_t at = w0; at < w1 && ok;) {
        const UnitPart x = unit_part(p.w, u, at, w1);
        const int n = x.j1 - x.j0, kvh = u.unit / p.row_blocks;
        at = x.next;
        if (n == 0) {
          if (at < w1) to_next();
          continue;
        }
        // Entries of the part's tiles i, i + 1, i + 2 (tile i is key tile j1 - 1 - i).
        const auto entry_of = [&](int i) { return i < n ? entry(x.j1 - 1 - i) : -1; };
        int e0 = entry_of(0), e1 = entry_of(1), e2 = entry_of(2);
        // The queries' place is free only when the last part's last scores have been
        // formed: keys first, but for the first part.
        const auto first_keys = [&]() {
          for (int i = 0; i < kAhead && i < n; ++i)
            fill(true, x.j1 - 1 - i, i ? e1 : e0, kvh, steps);
        };
        if (units > 0) {
          first_keys();
          if (keys) ok = ok && warp_wait(&bars.q_empty, (units - 1) & 1, bars.wait, a.status);
        }
        if (!ok) break;
        if (keys && leader) {
          const int nt = tiles_with_rows(u);
          const int node0 = (u.unit % p.row_blocks) * Shape::kQueryTiles * tp.tile_nodes;
          mbar_arrive_expect_tx(&bars.q, nt * tp.tile_rows * D * 2);
          for (int t = 0; t < nt; ++t)
            for (int b = 0; b < KB; ++b)
              tma_load_4d(smem + t * kTileBytes + b * kBlock, &tp.tq, b * 64, 0, kvh,
                          u.seq * a.n_new + node0 + t * tp.tile_nodes, &bars.q);
        }
        __syncwarp();
        if (units++ == 0) first_keys();
        for (int i = 0; i < n && ok; ++i) {
          fill(false, x.j1 - 1 - i, e0, kvh, steps + i);
          if (i + kAhead < n && ok)
            fill(true, x.j1 - 1 - i - kAhead, PAIR ? e1 : e2, kvh, steps + i);
          e0 = e1;
          e1 = e2;
          e2 = entry_of(i + 3);
        }
        steps += n;
        if (at < w1) to_next();
      }
      if (leader) {
        if (keys && units > 0) mbar_wait_bounded(&bars.q, (units - 1) & 1, a.status);
#pragma unroll
        for (int i = 0; i < kStages; ++i) bars.issued[warp - 1][i] = mine[i];
      }
    } else {
      // ---- products: the whole warp walks the loop, one elected lane issues
      bool ok = true;
      constexpr uint32_t kRowDesc = umma_idesc_bf16(kTileRows, D) | (1u << 16);  // B: N-major
      const uint64_t q_desc = umma_desc_sw128(smem_u32(smem));
      const uint64_t k_desc = umma_desc_sw128(smem_u32(ring));
      const uint64_t v_desc = umma_desc_rows(smem_u32(ring), kBlock);
      // S_t = Q K_jᵀ over `keys` keys, rounded up to 16.
      const auto issue_qk = [&](int t, int keys, int st) {
        const uint32_t idesc = umma_idesc_bf16(kTileRows, min(kTileRows, (keys + 15) & ~15));
        const uint64_t kd = k_desc + static_cast<uint32_t>(st * (kTileBytes >> 4));
        const uint64_t qd = q_desc + static_cast<uint32_t>(PAIR ? t * (kTileBytes >> 4) : 0);
        if (leader) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = ((ks >> 2) * kBlock + (ks & 3) * 32) >> 4;
            umma_bf16(tS[t], qd + off, kd + off, idesc, ks != 0);
          }
          umma_commit(&bars.s[t]);
        }
      };
      // O_t += P_t V_j over `keys` keys; `fresh`: the first step replaces O.
      const auto issue_pv = [&](int t, int keys, int st, bool fresh) {
        const uint64_t vd = v_desc + static_cast<uint32_t>(st * (kTileBytes >> 4));
        if (leader) {
          if (keys >= kTileRows) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              umma_bf16_ts(tO[t], tS[t] + ks * 8, vd + ks * (2048 >> 4), kRowDesc,
                           !(fresh && ks == 0));
          } else {
            for (int ks = 0; ks < (keys + 15) / 16; ++ks)
              umma_bf16_ts(tO[t], tS[t] + ks * 8, vd + ks * (2048 >> 4), kRowDesc,
                           !(fresh && ks == 0));
          }
        }
      };
      int st = 0;
      uint32_t parity = 0;
      // The next fill, once it has arrived.
      const auto arrived = [&]() {
        const int mine = st;
        ok = ok && warp_wait(&bars.full[st], parity, bars.wait, a.status);
        if (++st == kStages) {
          st = 0;
          parity ^= 1;
        }
        return mine;
      };
      uint32_t used[2] = {0, 0}, np[2] = {0, 0}, step = 0, units = 0;
      for (int64_t at = w0; at < w1 && ok;) {
        const UnitPart x = unit_part(p.w, u, at, w1);
        const int n = x.j1 - x.j0, nt = tiles_with_rows(u);
        at = x.next;
        if (n == 0) {
          if (at < w1) next_unit<MASK>(p.w, a.kv_len, u);
          continue;
        }
        const Span span = span_of<MASK>(p.w, u.len);
        const auto keys = [&](int i) { return tile_keys<MASK>(p.w, span, u.len, x.j1 - 1 - i); };
        ok = warp_wait(&bars.q, units++ & 1, bars.wait, a.status);
        for (int i = 0; i < kAhead && i < n && ok; ++i) {
          const int ks = arrived();
          if (!ok) break;
          tc_fence_after();
          if (PAIR) {
            for (int t = 0; t < nt; ++t) issue_qk(t, keys(0), ks);
          } else {
            issue_qk(i, keys(i), ks);
          }
        }
        if (ok && n <= kAhead && leader) umma_commit(&bars.q_empty);
        for (int i = 0; i < n && ok; ++i) {
          const int vs = arrived();
          const bool more = i + kAhead < n;
          const int ks = more ? arrived() : 0;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (PAIR ? t >= nt : t != (i & 1)) continue;
            const bool fresh = i < kAhead;
            if (fresh && used[t] > 0)
              ok = ok && warp_wait(&bars.o_empty[t], (used[t] - 1) & 1, bars.wait, a.status);
            ok = ok && warp_wait(&bars.p[t], np[t] & 1, bars.wait, a.status);
            if (!ok) continue;
            ++np[t];
            tc_fence_after();
            issue_pv(t, keys(i), vs, fresh);
            if (!more && leader) umma_commit(&bars.o[t]);
            if (!more) ++used[t];
            if (more) issue_qk(t, keys(i + kAhead), ks);
          }
          if (!ok) break;
          if (i + kAhead == n - 1 && leader) umma_commit(&bars.q_empty);
          if (leader) umma_commit(&bars.done[step & 7]);
          ++step;
        }
        if (at < w1) next_unit<MASK>(p.w, a.kv_len, u);
      }
      // Every product, and every arrival it still owes, ends before tensor
      // memory is freed and the CTA goes.
      if (leader) umma_commit(&bars.drain);
      __syncwarp();
      mbar_wait_bounded(&bars.drain, 0, a.status);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kUmmaSoftmaxRegs));
    // ---- softmax and output, one query row a thread
    const int t = (warp >> 2) - 1;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_addr = (t == 0 ? tS[0] : tS[1]) + lanes;
    const uint32_t o_addr = (t == 0 ? tO[0] : tO[1]) + lanes;
    const float mul = p.o.scale;  // unmapped scores enter the exponent as fma(s, mul, -m)
    int box_shift = 0;
    while ((1 << box_shift) < tp.box_rows) ++box_shift;
    const int kAllValid = (1 << (kTileRows / tp.box_rows)) - 1;
    uint32_t ns = 0, no[2] = {0, 0}, fills = 0, tiles = 0, units = 0;
    bool ok = true;
    for (int64_t at = w0; at < w1;) {
      const UnitPart x = unit_part(p.w, u, at, w1);
      const int n = x.j1 - x.j0, nt = tiles_with_rows(u);
      at = x.next;
      if (n == 0) {
        if (at < w1) next_unit<MASK>(p.w, a.kv_len, u);
        continue;
      }
      const int len = u.len, kvh = u.unit / p.row_blocks;
      const int row0 = (u.unit % p.row_blocks) * RT;
      // This thread's row: its node and head, whether it exists and has a node.
      const int r = row0 + (PAIR ? t * tp.tile_rows : 0) + row;
      const int rows = min(tp.tile_rows, g * a.n_new - row0 - (PAIR ? t * tp.tile_rows : 0));
      const bool there = row < rows;
      const int node = there ? r / g : 0, head = kvh * g + (there ? r - node * g : 0);
      const Span span = span_of<MASK>(p.w, len);
      // Tree: the ancestors of this row's node among the drafted rows, from `base`
      // on.  Window: the row sees keys from `low` up to `limit`, and the first ones.
      TreeNodes tree;
      uint64_t up = 0;
      int base = len, low = 0, limit = len, first_keys = 0, pos;
      bool live = there;
      if constexpr (MASK == kMaskTree) {
        // A part that ends before the drafted rows needs to know only how many there
        // are (a distance bias: their depths).
        base = len - tree.nodes(p.w, u.seq);
        tree.read(p.w, a, u.seq, lane, warp == 4, BIAS || x.j1 * kTileRows > base);
        live = there && node < tree.count;
        up = tree.ancestors(node);
        pos = base + tree.depth(node);
      } else {
        pos = len - a.n_new + node;
        if (there) {
          if (p.o.causal) limit = min(len, max(pos + 1, 0));
          low = pos - p.w.window + 1;
          first_keys = min(p.w.sinks, limit);
          if (!p.o.causal && p.w.window < len - pos) limit = pos + p.w.window;
        }
      }
      const bool warp_live = __any_sync(0xffffffffu, live);
      ScoreMap map;
      if (CAP || BIAS) {
        map.scale = pack2(p.o.scale, p.o.scale);
        constexpr float bend[5] = {kBend[0], kBend[1], kBend[2], kBend[3], kBend[4]};
        float unit = p.o.cap * p.o.scale;
#pragma unroll
        for (int i = 0; i < 5; ++i) {
          map.bend[i] = pack2(bend[i] * unit, bend[i] * unit);
          unit *= p.o.scale * p.o.scale;
        }
        map.weigh = live ? p.o.scale : 0.f;
        map.slope = BIAS ? load_input<kReadOrdered>(p.o.slopes + head) * kLog2e : 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          map.steps[i] = pack2(map.slope * (2 * i), map.slope * (2 * i + 1));
      }
      float m = -INFINITY, l = 0.f;
      for (int i = PAIR ? 0 : t; i < n && ok && t < (PAIR ? nt : 2); i += PAIR ? 1 : 2) {
        ok = warp_wait(&bars.s[t], ns & 1, bars.wait, a.status);
        if (!ok) break;
        ++ns;
        tc_fence_after();
        const int k0 = span.place(x.j1 - 1 - i) * kTileRows;
        const int valid = *reinterpret_cast<volatile int*>(&bars.valid[(tiles + i) & 7]);
        const bool edge =
            valid != kAllValid ||
            (MASK == kMaskTree
                 ? k0 + kTileRows > base
                 : __any_sync(0xffffffffu, k0 + kTileRows > limit || k0 < low));
        const bool first = PAIR ? i == 0 : i == t;
        const auto seen = [&](int c) {
          uint32_t bits = MASK == kMaskTree
                              ? tree_bits(up, k0 + c - base)
                              : seen_keys<true>(limit - k0 - c, low - k0 - c, first_keys - k0 - c);
          if (valid != kAllValid) bits &= box_bits(valid, c, box_shift);
          return bits;
        };
        uint64_t sum0 = 0, sum1 = 0;
        if (!warp_live) {
          // Rows without a node: their weights are never looked at.
        } else if constexpr (CAP || BIAS) {
          if (CAP && edge) {
            // Hidden scores become 0 in place (they may be NaN).
#pragma unroll 1
            for (int c = 0; c < 128; c += 32) {
              uint32_t w[32];
              tmem_ld32(s_addr + c, w);
              hide_keys(reinterpret_cast<float*>(w), seen(c), 0.f);
              tmem_st32(s_addr + c, w);
            }
            tmem_wait_st();
          }
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            uint32_t w[32], pk[16];
            tmem_ld32(s_addr + c, w);
            float* s = reinterpret_cast<float*>(w);
            const float d0 = static_cast<float>(pos - k0 - c);
            if (MASK == kMaskTree && BIAS && k0 + c + 32 > base) {
              // Drafted keys stand at their nodes' depths.
              if (CAP) map_scores<CAP, false>(s, p.o, map, d0, 1);
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const int key = k0 + c + e, depth = tree.depth(key - base);
                const int away = pos - (key < base ? key : base + depth);
                s[e] = fmaf(s[e], CAP ? 1.f : mul, -map.slope * fabsf(static_cast<float>(away)));
              }
            } else {
              // A tree's rows lie behind these keys.
              const int side = MASK == kMaskTree || !BIAS               ? 1
                               : __all_sync(0xffffffffu, d0 >= 31.f) ? 1
                               : __all_sync(0xffffffffu, d0 <= 0.f)  ? -1 : 0;
              map_scores<CAP, BIAS>(s, p.o, map, d0, side);
            }
            if (edge) hide_keys(s, seen(c));
            const float mc = chunk_max<32>(s);
            uint64_t add0, add1;
            while (true) {
              add0 = add1 = 0;
              chunk_weights<32>(s, 1.f, m, pk, add0, add1);
              if (__builtin_expect(!__any_sync(0xffffffffu, mc > m), 1)) break;
              // The sum, this tile's weights so far and O follow the maximum.
              float a0, a1;
              unpack2(add2(sum0, sum1), a0, a1);
              const float f = raise_max(m, mc, a0 + a1);
              if (f != 1.f) {
                l = (l + (a0 + a1)) * f;
                sum0 = sum1 = 0;
              }
              if (c > 0) tmem_wait_st();
              const __nv_bfloat162 fb = __float2bfloat162_rn(f);
#pragma unroll 1
              for (int e = 0; e < c / 2; e += 16) {
                uint32_t v[16];
                tmem_ld16(s_addr + e, v);
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                  const __nv_bfloat162 y =
                      __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v[k]), fb);
                  v[k] = *reinterpret_cast<const uint32_t*>(&y);
                }
                tmem_st16(s_addr + e, v);
              }
              if (!first) scale_output<D>(o_addr, f);
            }
            sum0 = add2(sum0, add0);
            sum1 = add2(sum1, add1);
            tmem_st16(s_addr + c / 2, pk);
          }
        } else {
          float mt = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 128; c += 64) {
            uint32_t w[64];
            tmem_ld64(s_addr + c, w);
            float* s = reinterpret_cast<float*>(w);
            if (edge) {
              hide_keys(s, seen(c));
              hide_keys(s + 32, seen(c + 32));
              tmem_st32(s_addr + c, w);
              tmem_st32(s_addr + c + 32, w + 32);
            }
            mt = fmaxf(mt, chunk_max<64>(s));
          }
          if (edge) tmem_wait_st();
          mt *= mul;
          if (first) {
            m = mt + kRaise;
          } else if (__any_sync(0xffffffffu, mt > m)) {
            const float f = raise_max(m, mt);
            l *= f;
            scale_output<D>(o_addr, f);
          }
#pragma unroll 1
          for (int c = 0; c < 128; c += 64) {
            uint32_t w[64], pk[32];
            tmem_ld64(s_addr + c, w);
            chunk_weights<64>(reinterpret_cast<const float*>(w), mul, m, pk, sum0, sum1);
            tmem_st32(s_addr + c / 2, pk);
          }
        }
        float a0, a1;
        unpack2(add2(sum0, sum1), a0, a1);
        l += a0 + a1;
        // Value rows behind the sequence's end, up to the product's, and those of
        // boxes without a page.
        const int rows_end = min(
            kTileRows, (tile_keys<MASK>(p.w, span, len, x.j1 - 1 - i) + 15) & ~15);
        if (len - k0 < rows_end || valid != kAllValid) {
          const uint32_t f = fills + (i < n - kAhead ? i + kAhead : n) + i;
          ok = warp_wait(&bars.full[f % kStages], (f / kStages) & 1, bars.wait, a.status);
          if (!ok) break;
          unsigned char* v = ring + (f % kStages) * kTileBytes;
          for (int e = row; e < rows_end * (D / 8); e += 128) {
            const int k = e / (D / 8), c = e % (D / 8);
            if (k0 + k < len && ((valid >> (k >> box_shift)) & 1)) continue;
            *reinterpret_cast<uint4*>(v + (c >> 3) * kBlock + k * 128 + (c & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async();
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars.p[t]);
      }
      // The fills' order: K_0 .. K_{L-1}, then V_i and K_{i+L}.
      fills += 2 * n;
      tiles += n;
      const bool two = !PAIR && n > 1;  // both groups have summed up keys
      if (PAIR ? t < nt : true) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (PAIR ? h != t : h == 1 && !two) continue;
          ok = ok && warp_wait(&bars.o[h], no[h] & 1, bars.wait, a.status);
          ++no[h];
        }
      }
      float f[2] = {1.f, 1.f};
      if (!PAIR) {
        // Both groups' sums, relative to the larger maximum (group 1 has none after a
        // single key tile).
        float(*ml)[kTileRows][2] = reinterpret_cast<float(*)[kTileRows][2]>(
            ring + kStages * kTileBytes + (units & 1) * (Shape::kSumBytes / 2));
        ml[t][row][0] = m;
        ml[t][row][1] = l;
        named_bar_sync(1, 256);  // also by a group that has given up
        m = fmaxf(ml[0][row][0], ml[1][row][0]);
        f[0] = m == -INFINITY ? 0.f : fast_exp2(ml[0][row][0] - m);
        f[1] = m == -INFINITY ? 0.f : fast_exp2(ml[1][row][0] - m);
        l = fmaf(f[1], ml[1][row][1], f[0] * ml[0][row][1]);
      }
      ++units;
      if (ok && (!PAIR || t < nt)) {
        tc_fence_after();
        if (!live) {
          m = -INFINITY;
          l = 0.f;
          f[0] = f[1] = 0.f;
        }
        const float inv = x.all ? inv_or_zero(l) : 1.f;
        // Four lanes write four rows together, 16 bytes of each in turn.
        const int row4 = row & ~3, part = lane & 3;
        const int64_t heads0 = static_cast<int64_t>(u.seq) * a.n_new * a.q_heads + kvh * g;
        float* slot = a.part + (2 * static_cast<int64_t>(blockIdx.x) + (u.begin >= w0 ? 1 : 0)) *
                                   RT * (D + 2);
        const int tile0 = PAIR ? t * tp.tile_rows : 0;  // first row within the block
        int place[4];  // rows of the output, relative to the sequence's
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int q = row0 + tile0 + row4 + j, i = q / g;
          place[j] = i * a.q_heads + (q - i * g);
        }
        constexpr int kMine = PAIR ? D : D / 2;  // columns of this group
        const int c0 = PAIR ? 0 : t * kMine;
#pragma unroll 1
        for (int c = c0; c < c0 + kMine; c += 32) {
          uint32_t o[32];
          float y[32];
          if (PAIR) {
            tmem_ld32(o_addr + c, o);
#pragma unroll
            for (int k = 0; k < 32; ++k) y[k] = __uint_as_float(o[k]) * inv;
          } else {
            tmem_ld32(tO[0] + lanes + c, o);
#pragma unroll
            for (int k = 0; k < 32; ++k) y[k] = __uint_as_float(o[k]) * (f[0] * inv);
            if (two) {
              tmem_ld32(tO[1] + lanes + c, o);
#pragma unroll
              for (int k = 0; k < 32; ++k) y[k] = fmaf(__uint_as_float(o[k]), f[1] * inv, y[k]);
            }
          }
          if (!live) {
#pragma unroll
            for (int k = 0; k < 32; ++k) y[k] = 0.f;
          }
          if (c == c0 + kMine - 32) {
            tc_fence_before();
            if (PAIR) {
              mbar_arrive(&bars.o_empty[t]);
            } else {
              mbar_arrive(&bars.o_empty[0]);
              if (two) mbar_arrive(&bars.o_empty[1]);
            }
          }
          uint32_t w[4][4];
          if (x.all) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * k], y[2 * k + 1]);
              w[k / 4][k % 4] = *reinterpret_cast<const uint32_t*>(&b);
            }
            exchange_rows(w, part);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (row4 + j < rows)
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) +
                                          (heads0 + place[j]) * D + c + 8 * part) =
                    make_uint4(w[j][0], w[j][1], w[j][2], w[j][3]);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int k = 0; k < 16; ++k) w[k / 4][k % 4] = __float_as_uint(y[16 * h + k]);
              exchange_rows(w, part);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (row4 + j < rows)
                  *reinterpret_cast<uint4*>(slot + static_cast<int64_t>(tile0 + row4 + j) * D + c +
                                            16 * h + 4 * part) =
                      make_uint4(w[j][0], w[j][1], w[j][2], w[j][3]);
            }
          }
        }
        if (there && (PAIR || t == 0)) {
          if (!x.all)
            *reinterpret_cast<float2*>(slot + static_cast<int64_t>(RT) * D + 2 * (tile0 + row)) =
                make_float2(m, l);
          else if (a.lse != nullptr)
            a.lse[heads0 + node * a.q_heads + head - kvh * g] = row_lse(m, l);
        }
      }
      if (at < w1) next_unit<MASK>(p.w, a.kv_len, u);
    }
  }
  __syncwarp();  // the issuing lanes rejoin their warps
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
  // Nothing of this CTA's copies may land after it has gone, also where a role has
  // given up before their products.  A stage's last fill only: what either warp
  // issued before it had been used, and its barrier has moved on.
  if (threadIdx.x < kStages) {
    const uint32_t last = max(bars.issued[0][threadIdx.x], bars.issued[1][threadIdx.x]);
    if (last > 0)
      mbar_wait_bounded(&bars.full[threadIdx.x], ((last - 1) / kStages) & 1, a.status);
  }
}

template <int D, bool PAIR, int MASK, bool CAP, bool BIAS>
cudaError_t launch_umma(const UmmaParams& p, const PagedPlan& plan, cudaStream_t stream) {
  const cudaError_t e = ensure_max_smem<paged_umma_kernel<D, PAIR, MASK, CAP, BIAS>>();
  if (e != cudaSuccess) return e;
  return launch_early(paged_umma_kernel<D, PAIR, MASK, CAP, BIAS>, dim3(plan.ctas), kUmmaThreads,
                      UmmaShape<D, PAIR>::kSmem, stream, p);
}

template <int D, bool PAIR, int MASK>
cudaError_t launch_umma_opts(const UmmaParams& p, const PagedPlan& plan, cudaStream_t stream) {
  const bool bias = p.p.o.slopes != nullptr;
  if (p.p.o.cap > 0.f)
    return bias ? launch_umma<D, PAIR, MASK, true, true>(p, plan, stream)
                : launch_umma<D, PAIR, MASK, true, false>(p, plan, stream);
  return bias ? launch_umma<D, PAIR, MASK, false, true>(p, plan, stream)
              : launch_umma<D, PAIR, MASK, false, false>(p, plan, stream);
}

template <int D, int MASK>
cudaError_t launch_umma_dim(const PagedArgs& a, const PagedPlan& plan, cudaStream_t stream) {
  UmmaParams p;
  const int g = a.q_heads / a.kv_heads;
  p.p = paged_params(a, plan);
  p.box_rows = std::min(a.page_size, kTileRows);
  p.page_shift = 0;
  while ((1 << p.page_shift) < a.page_size) ++p.page_shift;
  p.tile_nodes = kTileRows / g;
  p.tile_rows = p.tile_nodes * g;
  p.inject_polls = consume_wait_injection();
  const cuuint64_t d = D, row = D * 2;
  // Queries: channels, heads of a key-value head, key-value heads, nodes.
  const cuuint64_t q_dims[4] = {d, static_cast<cuuint64_t>(g), static_cast<cuuint64_t>(a.kv_heads),
                                static_cast<cuuint64_t>(a.n_seqs) * a.n_new};
  const cuuint64_t q_strides[3] = {row, row * g, row * a.q_heads};
  const cuuint32_t q_box[4] = {64, static_cast<cuuint32_t>(g), 1,
                               static_cast<cuuint32_t>(p.tile_nodes)};
  const cuuint64_t dims[2] = {d, static_cast<cuuint64_t>(a.n_pages) * a.kv_heads * a.page_size};
  const cuuint64_t strides[1] = {row};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(p.box_rows)};
  constexpr CUtensorMapDataType kType = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (!encode_tile_map(&p.tq, kType, a.q, 4, q_dims, q_strides, q_box) ||
      !encode_tile_map(&p.tk, kType, a.k_pages, 2, dims, strides, box) ||
      !encode_tile_map(&p.tv, kType, a.v_pages, 2, dims, strides, box))
    return cudaErrorInvalidValue;
  const cudaError_t e = a.n_new > p.tile_nodes ? launch_umma_opts<D, true, MASK>(p, plan, stream)
                                               : launch_umma_opts<D, false, MASK>(p, plan, stream);
  return e != cudaSuccess ? e : launch_join<__nv_bfloat16, D, MASK>(a, plan, stream);
}

// More rows than this a key head run here (bf16; groups of up to 128 heads, a node
// of which fits a tile).  Up to four rows the warps of the other kernel add up in
// one go: trees over four sequences of 300 to 1500 keys 14.6 us against 18 here,
// but 24.8 against 18.9 for 16 rows; 16 sequences of 6800 keys 87 against 83.
constexpr int kFewRows = 4;
// What a unit costs its CTA beside its tiles (queries, output, the gap in the
// products and in its copies), in tiles.  Trees of 26 nodes over 16 sequences of 1000
// to 16384 keys: 101 us without, 96, 93, 90, 88, 88 with 1 to 5; of 64 nodes over 24 of
// 540 to 25890 keys: 232 without, 216, 205, 196 with 1 to 3, 199 with 5.
constexpr int kPadOne = 4, kPadPair = 3;
inline bool on_umma(const PagedArgs& a) {
  const int g = a.q_heads / a.kv_heads;
  return a.dtype == WF_BF16 && g <= kTileRows && g * a.n_new > kFewRows;
}

inline PagedPlan plan_umma(const PagedArgs& a, int sm_count) {
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

template <int MASK>
cudaError_t launch_umma_mask(const PagedArgs& a, const PagedPlan& plan, cudaStream_t stream) {
  return a.head_dim == 128 ? launch_umma_dim<128, MASK>(a, plan, stream)
                           : launch_umma_dim<64, MASK>(a, plan, stream);
}

}  // namespace

}  // namespace wf
