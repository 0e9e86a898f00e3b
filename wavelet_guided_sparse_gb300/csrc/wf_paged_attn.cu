// Attention of new tokens over a paged key-value cache (eq. (3) over the
// whole cache): the split kernel, the join of split sequences, plan and
// dispatch.
//
// HBM-bound at bf16 while all g n_new query rows that share a key head fit one
// row block of at most 64: each key-value row is then read once (16 to 64 flop
// a byte), and everything serves the stream.  More rows read it once a block.
// The 64-key tiles of all sequences and heads form one line that a
// persistent grid divides evenly (wf_attn.cuh).  In each CTA one producer
// warp keeps a ring of tiles full by tensor copies (whole pages, or 64-row
// parts of them, 128-byte swizzle), reading the page table one tile ahead;
// the consumer warps hold 16 query rows each and split a tile's keys:
//   rows <= 16: 4 warps x 16 keys, two CTAs an SM (3 stages of 32 KB each);
//               fp32: 8 warps x 8 keys, one CTA, 3 stages of 64 KB;
//   rows <= 32: 2 row tiles x 4 warps x 16 keys, one CTA, 6 stages (fp32: 3);
//   otherwise : 4 row tiles x 2 warps x 32 keys, one CTA, 5 stages (fp32: 2).
// The products are mma.sync m16n8k16 (bf16 in, fp32 accumulate): at 16 rows a
// 128-row tcgen05 tile would be seven eighths empty, and the pipe is far
// from the bound.  Every warp keeps its own running (max, sum, O) over its
// keys, in weights of at most 1 (a value of the type's largest must not
// overflow on the way); the maximum is raised lazily: 8 (in log2; fp32: 1)
// above the score that raised it, so that only a score beyond that raises it
// again.  The warps of a row tile add up once per unit, in a fixed order.
//
// fp32 operands meet the tensor cores as two tf32 parts each (x = hi + lo to
// 2^-22, and no finer than 2^-137; hi hi + hi lo + lo hi): the error of a
// product stays below 2^-20 |a||b|, the order of the fp32 sums around it.
//
// Rows behind a sequence's end (the tail of its last page, stale stages) and
// rows of bad pages get weights of exactly 0 and their value rows are
// cleared in shared memory before the product.
//
// Measured (32 query heads, d = 128; the stream's share of the measured copy
// rate).  8 heads of keys, one new token: 64 sequences of 200 to 16384 keys
// 146 to 148 us, 89 %; one of 131072 keys with capped scores or a bias 87 us,
// 91 %.  32 heads of keys, a block of 32 tokens, two sequences of 65536 keys:
// 324 us, 98 %.  The same block over 8 heads of keys (128 rows, two row blocks),
// 16 sequences of 8192 keys: 238 us, 33 % of one read.
// A few hundred keys: 14 us, of which the split kernel's code, tables and
// first tile take 9 and the join 5.  fp32, 16 sequences of 8192 keys: 320 us,
// 49 %, bound by the tf32 products (the FMA pipes took 783).
#include <algorithm>

#include "wf_attn.cuh"
#include "wf_mma.cuh"
#include "wf_tensormap.h"
#include "wf_umma.cuh"

namespace wf {

namespace {

constexpr int KT = kPagedTile;  // keys per tile
// What a raised maximum is set above the score that raised it (log2).  fp32: 1,
// since the exponents' arguments round in proportion to their size.
template <typename T>
constexpr float kHeadroom = sizeof(T) == 2 ? 8.f : 1.f;

// An fp32 word as two tf32 parts, x = hi + lo to 2^-22 relative.  FINITE: hi
// stays finite, whatever x.  The largest numbers keep their rest in lo, and an
// infinity is lo alone, so that of its products only that with the other
// operand's hi, which has that operand's sign, is infinite (an infinite hi
// would meet lo's of either sign, or 0).
template <bool FINITE>
__device__ __forceinline__ void split_tf32(uint32_t x, uint32_t& hi, uint32_t& lo) {
  if (FINITE)
    asm("cvt.rna.satfinite.tf32.f32 %0, %1;" : "=r"(hi) : "f"(__uint_as_float(x)));
  else
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(__uint_as_float(x)));
  const float rest = __uint_as_float(x) - __uint_as_float(hi);
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(rest));
}
// Two weights (not negative) as two bf16 parts each, x = hi + lo to 2^-15.  hi
// is cut, so that lo is not negative, and lo is never 0 beside hi: both meet an
// infinite value with its sign.
__device__ __forceinline__ void split_weights(float x, float y, uint32_t& hi, uint32_t& lo) {
  const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
  hi = __byte_perm(a, b, 0x7632);
  lo = pack_bf16(fmaxf(x - __uint_as_float(a & 0xffff0000u), x * 0x1p-20f),
                 fmaxf(y - __uint_as_float(b & 0xffff0000u), y * 0x1p-20f));
}
// D = A(16x8, row) * B(8x8, col) + D; tf32 inputs, fp32 accumulators.
__device__ __forceinline__ void mma_tf32(float* c, const uint32_t* a, const uint32_t* b) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// R: 16-row query tiles per CTA.
template <typename T, int D, int R>
struct PagedShape {
  static constexpr bool kWide = sizeof(T) == 4;         // fp32: twice the bytes a tile
  static constexpr int kConsumers = R == 1 && !kWide ? 4 : 8;  // warps
  static constexpr int kKeyGroups = kConsumers / R;
  static constexpr int kKeys = KT / kKeyGroups;         // keys per warp and tile
  static constexpr int kThreadCount = (kConsumers + 1) * 32;
  static constexpr int kCtasPerSm = kConsumers == 4 ? 2 : 1;
  static constexpr int kTileBytes = KT * D * static_cast<int>(sizeof(T));  // keys or values
  static constexpr int kStages =
      (kWide ? (R == 4 ? 2 : 3) : R == 1 ? 3 : R == 2 ? 6 : 5) * (D == 64 ? 2 : 1);
  static constexpr int kPitch = D + 4;                  // floats per merge row
  static constexpr int kMergeRows = R == 1 ? 4 * kConsumers : 16 * R;
  static constexpr int kQueryBytes = 16 * R * D * static_cast<int>(sizeof(T));
  static constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * 2 * kTileBytes +
                                  kMergeRows * kPitch * sizeof(float) + kQueryBytes;
};

struct PagedTcParams {
  CUtensorMap tk, tv;
  PagedParams p;
  int box_rows, page_shift;
  uint32_t inject_polls;  // fault injection (tests): see the kernel's start
};

template <int STAGES>
struct PagedBarriers {
  uint64_t full[STAGES], empty[STAGES], q_empty;
  int valid[STAGES];  // one bit per box of a stage
  WaitState wait;
};

template <typename T, int D, int R, bool CAP, bool BIAS>
__global__ void
__launch_bounds__(PagedShape<T, D, R>::kThreadCount, PagedShape<T, D, R>::kCtasPerSm)
    paged_tc_kernel(const __grid_constant__ PagedTcParams tp) {
  using Shape = PagedShape<T, D, R>;
  constexpr bool kWide = Shape::kWide;
  constexpr int kStages = Shape::kStages, kTileBytes = Shape::kTileBytes;
  constexpr int kStageBytes = 2 * kTileBytes, RT = 16 * R;
  constexpr int kConsumerThreads = Shape::kConsumers * 32;
  // fp32: first parts that are always finite.  They cost a 16-row unit, whose
  // queries are split again every 8 keys, 8 % (16 sequences of 8192 keys: 345 us
  // against 319), more rows 1 to 6 %, less than the other way, below, would.
  constexpr bool kFinite = R > 1;
  constexpr int KC = 128 / sizeof(T), KB = D / KC;  // columns of a 128-byte block, blocks of a row
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) PagedBarriers<kStages> bars;
  __shared__ float s_ml[Shape::kKeyGroups][RT][2];
  unsigned char* ring = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* merge = reinterpret_cast<float*>(ring + kStages * kStageBytes);
  T* s_q = reinterpret_cast<T*>(merge + Shape::kMergeRows * Shape::kPitch);
  const PagedParams& p = tp.p;
  const PagedArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = a.q_heads / a.kv_heads;

  // Fault injection (tests of the bounded waits): the first CTA's first tile is
  // never issued, and its waits give up after inject_polls polls.
  const bool inject = tp.inject_polls != 0 && blockIdx.x == 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.empty[i], Shape::kConsumers);
    }
    mbar_init(&bars.q_empty, Shape::kConsumers);
    bars.wait.init(inject ? tp.inject_polls : kWaitPolls);
    fence_mbar_init();
  }
  const WorkSplit split(work_total(p.w, a.kv_len), gridDim.x);
  const int64_t w0 = split.begin(blockIdx.x), w1 = split.begin(blockIdx.x + 1);
  WorkUnit u = find_unit(p.w, a.kv_len, w0);
  __syncthreads();
  launch_dependents();

  if (warp == Shape::kConsumers) {
    // ---- producer: lane = (box of the stage, keys or values, column block);
    // where a stage has more than 32 such parts, a lane has NS of them
    const int boxes = KT / tp.box_rows;
    constexpr int NS = KB > 2 ? 2 : 1, kSubs = 32 / (2 * KB);
    const int kb = lane % KB, which = (lane / KB) & 1, sub = lane / (2 * KB);
    const uint32_t box_bytes = static_cast<uint32_t>(tp.box_rows) * 128;
    const CUtensorMap* map = which ? &tp.tv : &tp.tk;
    if (lane == 0) {
      prefetch_tensormap(&tp.tk);
      prefetch_tensormap(&tp.tv);
    }
    // Page-table entries of this lane's boxes of a tile (-1: nothing to copy),
    // only looked at when their copies are issued: the loads fly meanwhile.
    int page[NS];
    const auto read_entries = [&](const WorkUnit& x, int64_t at) {
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int box = sub + i * kSubs;
        const int key = static_cast<int>(at - x.begin) * KT + box * tp.box_rows;
        page[i] = -1;
        if (box < boxes && key < x.len)
          page[i] = __ldg(a.table + static_cast<int64_t>(x.seq) * a.table_pages +
                          (key >> tp.page_shift));
      }
    };
    unsigned every[NS];  // the lanes with a part of a full stage
#pragma unroll
    for (int i = 0; i < NS; ++i) every[i] = __ballot_sync(0xffffffffu, sub + i * kSubs < boxes);
    int fill = 0, units = 0, st = 0;
    uint32_t phase = 1;  // of the stage's last release (first time: none yet)
    int row0 = 0, rows = 0, kvh = 0;
    bool ok = true;
    if (w0 < w1) read_entries(u, w0);
    for (int64_t at = w0; at < w1; ++at) {
      // A unit's query rows arrive with its first tile: the runs of rows that
      // one query's heads (or a part of them) form, one bulk copy each.
      const bool first = at == w0 || at == u.begin;
      if (first) {
        kvh = u.unit / p.row_blocks;
        row0 = (u.unit - kvh * p.row_blocks) * RT;
        rows = min(RT, g * a.n_new - row0);
        if (units++ > 0) {
          ok = warp_wait(&bars.q_empty, (units - 2) & 1, bars.wait, a.status);
          if (!ok) break;
        }
      }
      if (fill >= kStages) {
        ok = warp_wait(&bars.empty[st], phase, bars.wait, a.status);
        if (!ok) break;
      }
      const int key0 = static_cast<int>(at - u.begin) * KT;
      unsigned live[NS];
      int parts = 0;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int box = sub + i * kSubs;
        if (page[i] < 0 || page[i] >= a.n_pages) {
          if (box < boxes && key0 + box * tp.box_rows < u.len)
            raise_flag(a.status, WF_DEV_BAD_INDEX);
          page[i] = -1;
        }
        live[i] = __ballot_sync(0xffffffffu, page[i] >= 0);
        parts += __popc(live[i]);
      }
      const bool issue = !(inject && fill == 0);
      if (lane == 0 && issue) {
        int valid = (1 << boxes) - 1;
#pragma unroll
        for (int i = 0; i < NS; ++i)
          if (live[i] != every[i])
            for (int e = 0; e < kSubs; ++e)
              if (!((live[i] >> (e * 2 * KB)) & 1)) valid &= ~(1 << (i * kSubs + e));
        bars.valid[st] = valid;
        mbar_arrive_expect_tx(&bars.full[st],
                              parts * box_bytes +
                                  (first ? rows * D * static_cast<int>(sizeof(T)) : 0));
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        if (page[i] < 0 || !issue) continue;
        const int box = sub + i * kSubs, key = key0 + box * tp.box_rows;
        const int y = (page[i] * a.kv_heads + kvh) * a.page_size + (key & (a.page_size - 1));
        tma_load_2d(ring + st * kStageBytes + which * kTileBytes + kb * (KT * 128) +
                        box * box_bytes,
                    map, kb * KC, y, &bars.full[st]);
      }
      if (first && issue) {
        const int i0 = row0 / g, i1 = (row0 + rows - 1) / g;
        for (int i = i0 + lane; i <= i1; i += 32) {
          const int r0 = max(i * g, row0), r1 = min((i + 1) * g, row0 + rows);
          const int64_t from = (static_cast<int64_t>(u.seq) * a.n_new + i) * a.q_heads + kvh * g +
                               (r0 - i * g);
          bulk_g2s(s_q + (r0 - row0) * D, static_cast<const T*>(a.q) + from * D,
                   (r1 - r0) * D * static_cast<int>(sizeof(T)), &bars.full[st]);
        }
      }
      ++fill;
      if (++st == kStages) {
        st = 0;
        phase ^= 1;
      }
      if (at + 1 < w1) {
        if (at + 1 == u.begin + u.tiles) next_unit(p.w, a.kv_len, u);
        read_entries(u, at + 1);
      }
    }
    // No copy may land after the CTA has gone, also where the consumers have
    // given up behind this warp's last wait.
    for (int f = max(inject ? 1 : 0, fill - kStages); f < fill; ++f)
      mbar_wait_bounded(&bars.full[f % kStages], (f / kStages) & 1, a.status);
  } else {
    // ---- consumers
    const int rt = warp % R, kg = warp / R;      // row tile, key group
    const int gid = lane >> 2, tig = lane & 3;
    idle_sequences<T>(a, p.w.max_len, blockIdx.x, gridDim.x, threadIdx.x,
                                  kConsumerThreads);
    // Scores enter the exponent as fma(s, mul, -m); biased ones are whole before.
    const float unit = CAP ? p.o.cap : p.o.scale, mul = BIAS ? 1.f : unit;
    // ldmatrix lane addresses within a tile: keys as B (rows = keys), values
    // transposed (rows = keys); 16-byte chunk c of row r sits at c ^ (r % 8),
    // so a step along a row is an exclusive or of bits 5-6 (and a column
    // block every four).
    // fp32: an ldmatrix reads four 16-byte chunks of eight keys (two steps of 8
    // channels); a weight's register pair (keys 2 tig, 2 tig + 1) is taken as
    // rows tig and tig + 4 of the product, so values come as words of rows
    // 2 tig and 2 tig + 1, whose chunks lie in different banks.
    const int krow = kg * Shape::kKeys + (kWide ? 0 : (lane >> 4) << 3) + (lane & 7);
    const int vrow = kg * Shape::kKeys + (kWide ? 2 * tig : (((lane >> 3) & 1) << 3) + (lane & 7));
    const uint32_t koff =
        krow * 128 + (((kWide ? lane >> 3 : (lane >> 3) & 1) ^ (krow & 7)) << 4);
    const uint32_t voff = kWide ? vrow * 128 + (((gid >> 2) ^ (vrow & 7)) << 4) + (gid & 3) * 4
                                : vrow * 128 + (((lane >> 4) ^ (vrow & 7)) << 4);
    const uint32_t ring_addr = smem_u32(ring);
    const int kAllValid = (1 << (KT / tp.box_rows)) - 1;
    int st = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int64_t at = w0; at < w1;) {
      const int64_t end = min(w1, u.begin + u.tiles);
      const int len = u.len;
      const int prefix = p.o.prefix != nullptr ? __ldg(p.o.prefix + u.seq) : 0;
      const int kvh = u.unit / p.row_blocks;
      const int row0 = (u.unit % p.row_blocks) * RT;
      const int rows = min(RT, g * a.n_new - row0);
      const int64_t base = static_cast<int64_t>(u.seq) * a.n_new * a.q_heads + kvh * g;
      // This lane's two query rows: position, key limit, slope.
      int pos[2], limit[2];
      float slope[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = row0 + rt * 16 + gid + 8 * h;
        const bool live = r - row0 < rows;
        const int i = live ? r / g : 0, hd = live ? r - i * g : 0;
        pos[h] = len - a.n_new + i;
        limit[h] = p.o.causal ? min(len, max(pos[h] + 1, prefix)) : len;
        slope[h] = BIAS ? __ldg(p.o.slopes + kvh * g + hd) * kLog2e : 0.f;
      }
      // The unit's query rows arrive with its first tile.
      ok = ok && warp_wait(&bars.full[st], phase, bars.wait, a.status);
      constexpr int KS = D * static_cast<int>(sizeof(T)) / 32;  // steps of a score's product
      constexpr int kHalf = 16 / static_cast<int>(sizeof(T));   // channels of half a step
      uint32_t qf[KS][4];
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int r = rt * 16 + gid + 8 * (c & 1);
          qf[ks][c] = r < rows ? *reinterpret_cast<const uint32_t*>(
                                     s_q + r * D + (2 * ks + (c >> 1)) * kHalf + tig * (kHalf / 4))
                               : 0u;
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.q_empty);
      float o[D / 8][4];
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

      const int tiles = static_cast<int>(end - at);
      int key0 = static_cast<int>(at - u.begin) * KT + kg * Shape::kKeys;
      at = end;
      // Keys below `open` are visible to every row of the warp.
      int open = min(limit[0], limit[1]);
#pragma unroll
      for (int w = 4; w < 32; w <<= 1) open = min(open, __shfl_xor_sync(0xffffffffu, open, w));
      for (int i = 0; i < tiles; ++i, key0 += KT) {
        ok = ok && warp_wait(&bars.full[st], phase, bars.wait, a.status);
        if (!ok) break;  // given up: only the barriers below, in step with the other warps
        const uint32_t kt = ring_addr + st * kStageBytes + koff;
        const uint32_t vt = ring_addr + st * kStageBytes + kTileBytes + voff;
        const int valid = *reinterpret_cast<volatile int*>(&bars.valid[st]);
        const bool edge = valid != kAllValid || key0 + Shape::kKeys > open;
        if (edge && (valid != kAllValid || key0 + Shape::kKeys > len)) {
          // Clear the value rows whose weight is 0 by their place (and the keys
          // where a score that is not finite would choose the form of the tile's).
          constexpr int C = D * static_cast<int>(sizeof(T)) / 16;  // chunks of a row
          for (int e = lane; e < Shape::kKeys * C; e += 32) {
            const int r = e / C, c = e % C;
            const int tr = kg * Shape::kKeys + r;
            if (key0 + r >= len || !((valid >> (tr / tp.box_rows)) & 1)) {
              uint4* chunk = reinterpret_cast<uint4*>(ring + st * kStageBytes + (c >> 3) * (KT * 128) +
                                                      tr * 128 + (c & 7) * 16);
              chunk[kTileBytes / 16] = make_uint4(0u, 0u, 0u, 0u);
              if (kWide && !kFinite) *chunk = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          fence_proxy_async();
          __syncwarp();
        }
        constexpr int NB = Shape::kKeys / 8;  // 8-key blocks
        // Two accumulators a block halve the chain of dependent products; for
        // fp32 the second one takes the small terms.
        float s[NB][4], s2[NB][4];
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] = s2[n][e] = 0.f;
        if constexpr (kWide) {
#pragma unroll
          for (int j = 0; j < KS / 2; ++j) {
            uint32_t qh[2][4], ql[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int c = 0; c < 4; ++c) split_tf32<kFinite>(qf[2 * j + h][c], qh[h][c], ql[h][c]);
#pragma unroll
            for (int n = 0; n < NB; ++n) {
              uint32_t b[4], bh[4], bl[4];
              ldsm_x4((kt ^ ((j & 1) << 6)) + (j >> 1) * (KT * 128) + n * 1024, b);
#pragma unroll
              for (int e = 0; e < 4; ++e) split_tf32<kFinite>(b[e], bh[e], bl[e]);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                mma_tf32(s[n], qh[h], bh + 2 * h);
                mma_tf32(s2[n], qh[h], bl + 2 * h);
                mma_tf32(s2[n], ql[h], bh + 2 * h);
              }
            }
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
#pragma unroll
            for (int n = 0; n < NB; n += 2) {
              uint32_t b[4];
              ldsm_x4((kt ^ ((ks & 3) << 5)) + (ks >> 2) * (KT * 128) + n * 1024, b);
              mma_bf16(ks & 1 ? s2[n] : s[n], qf[ks], b);
              mma_bf16(ks & 1 ? s2[n + 1] : s[n + 1], qf[ks], b + 2);
            }
          }
        }
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] += s2[n][e];
        if constexpr (kWide && !kFinite) {
          // A score that is not finite shows operands whose first part may not be
          // (infinities, the largest numbers): once more, by fp32 products.
          bool odd = false;
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) odd |= !(fabsf(s[n][e]) < INFINITY);
          if (__builtin_expect(__any_sync(0xffffffffu, odd), 0)) {
            const float* row[2];  // this lane's query rows (dead ones: the unit's first)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int r = rt * 16 + gid + 8 * h < rows ? row0 + rt * 16 + gid + 8 * h : row0;
              row[h] = static_cast<const float*>(a.q) +
                       (base + static_cast<int64_t>(r / g) * a.q_heads + r % g) * D;
            }
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int r = kg * Shape::kKeys + n * 8 + 2 * tig + (e & 1);
                const unsigned char* key = ring + st * kStageBytes + r * 128;
                float sum = 0.f;
#pragma unroll 1
                for (int c = 0; c < D / 4; ++c) {
                  const float4 x = *reinterpret_cast<const float4*>(
                      key + (c >> 3) * (KT * 128) + (((c & 7) ^ (r & 7)) << 4));
                  const float4 y = __ldg(reinterpret_cast<const float4*>(row[e >> 1]) + c);
                  sum = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, sum))));
                }
                s[n][e] = sum;
              }
          }
        }
        if (CAP) {
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] = tanh_exp2(s[n][e] * p.o.scale);
        }
        if (BIAS) {
          // Distances from the tile's first key as whole numbers: positions past
          // 2^24 do not fit fp32, the distances that weigh anything do.
          const float d0[2] = {static_cast<float>(pos[0] - key0 - 2 * tig),
                               static_cast<float>(pos[1] - key0 - 2 * tig)};
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              s[n][e] = fmaf(s[n][e], unit, -slope[e >> 1] *
                             fabsf(d0[e >> 1] - static_cast<float>(n * 8 + (e & 1))));
        }
        if (edge) {
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int r = n * 8 + 2 * tig + (e & 1);
              const bool there = (valid >> ((kg * Shape::kKeys + r) / tp.box_rows)) & 1;
              s[n][e] = there && key0 + r < limit[e >> 1] ? s[n][e] : -INFINITY;
            }
        }
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          mx[0] = fmaxf(mx[0], fmaxf(s[n][0], s[n][1]));
          mx[1] = fmaxf(mx[1], fmaxf(s[n][2], s[n][3]));
        }
        // A row's lanes must agree on its maximum; whether any has grown too
        // far, every lane can tell from its own part.
        if (__any_sync(0xffffffffu, mx[0] * mul > m[0] || mx[1] * mul > m[1])) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2)) * mul;
            const float mn = mx[h] > m[h] ? mx[h] + kHeadroom<T> : m[h];
            const float f = mn == -INFINITY ? 1.f : fast_exp2(m[h] - mn);
            m[h] = mn;
            l[h] *= f;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
              o[n][2 * h] *= f;
              o[n][2 * h + 1] *= f;
            }
          }
        }
        const float b0 = m[0] == -INFINITY ? 0.f : m[0], b1 = m[1] == -INFINITY ? 0.f : m[1];
        // Up to 16 rows the tensor cores are idle enough to take bf16's weights in
        // two parts (1 % more time: 131072 keys 86.5 -> 87.5 us; relative error of
        // the output 0.0024 -> 0.0017, that of its own rounding).  More rows take
        // them rounded to bf16, half a step, 2^-8 relative each: two parts would
        // cost 32 tokens over 2 x 65536 keys 325 -> 354 us.
        constexpr bool kTwoParts = !kWide && R == 1;
        uint32_t pf[NB][kWide ? 4 : 2], pl[kTwoParts ? NB : 1][2];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          const float e0 = fast_exp2(fmaf(s[n][0], mul, -b0)), e1 = fast_exp2(fmaf(s[n][1], mul, -b0));
          const float e2 = fast_exp2(fmaf(s[n][2], mul, -b1)), e3 = fast_exp2(fmaf(s[n][3], mul, -b1));
          l[0] += e0 + e1;
          l[1] += e2 + e3;
          if constexpr (kWide) {
            pf[n][0] = __float_as_uint(e0);
            pf[n][1] = __float_as_uint(e2);
            pf[n][2] = __float_as_uint(e1);
            pf[n][3] = __float_as_uint(e3);
          } else if constexpr (kTwoParts) {
            split_weights(e0, e1, pf[n][0], pl[n][0]);
            split_weights(e2, e3, pf[n][1], pl[n][1]);
          } else {
            pf[n][0] = pack_bf16(e0, e1);
            pf[n][1] = pack_bf16(e2, e3);
          }
        }
        if constexpr (kWide) {
#pragma unroll
          for (int kk = 0; kk < NB; ++kk) {
            uint32_t ah[4], al[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) split_tf32<false>(pf[kk][e], ah[e], al[e]);
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
              // Rows 2 tig and 2 tig + 1: the odd row's chunk is the even one's
              // neighbour in its pair.
              const uint32_t at = (vt ^ ((n & 3) << 5)) + (n >> 2) * (KT * 128) + kk * 1024;
              uint32_t bh[2], bl[2];
              split_tf32<true>(lds32(at), bh[0], bl[0]);
              split_tf32<true>(lds32((at ^ 16) + 128), bh[1], bl[1]);
              mma_tf32(o[n], ah, bl);
              mma_tf32(o[n], al, bh);
              mma_tf32(o[n], ah, bh);
            }
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < NB / 2; ++kk) {
            const uint32_t af[4] = {pf[2 * kk][0], pf[2 * kk][1], pf[2 * kk + 1][0], pf[2 * kk + 1][1]};
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
              uint32_t b[4];
              ldsm_x4_t((vt ^ ((n & 3) << 5)) + (n >> 2) * (KT * 128) + kk * 2048, b);
              if constexpr (kTwoParts) {
                const uint32_t al[4] = {pl[2 * kk][0], pl[2 * kk][1], pl[2 * kk + 1][0],
                                        pl[2 * kk + 1][1]};
                mma_bf16(o[2 * n], al, b);
                mma_bf16(o[2 * n + 1], al, b + 2);
              }
              mma_bf16(o[2 * n], af, b);
              mma_bf16(o[2 * n + 1], af, b + 2);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.empty[st]);
        if (++st == kStages) {
          st = 0;
          phase ^= 1;
        }
      }

      // The warps of a row tile add up, in key-group order: every warp leaves
      // its O (relative to its own maximum) in a slot of the merge buffer,
      // all slots at once where the unit's rows leave room, else one group
      // after the other.
      const bool at_once = rows * Shape::kKeyGroups <= Shape::kMergeRows;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      }
      named_bar_sync(1, kConsumerThreads);  // the last unit's output has left the buffer
      if (tig == 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          s_ml[kg][rt * 16 + gid + 8 * h][0] = m[h];
          s_ml[kg][rt * 16 + gid + 8 * h][1] = l[h];
        }
      }
      if (at_once) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = rt * 16 + gid + 8 * h;
          if (r < rows) {
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
              *reinterpret_cast<float2*>(merge + (kg * rows + r) * Shape::kPitch + n * 8 + 2 * tig) =
                  make_float2(o[n][2 * h], o[n][2 * h + 1]);
          }
        }
      } else {
        named_bar_sync(1, kConsumerThreads);
        float f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = rt * 16 + gid + 8 * h;
          float gm = -INFINITY;
#pragma unroll
          for (int k = 0; k < Shape::kKeyGroups; ++k) gm = fmaxf(gm, s_ml[k][r][0]);
          f[h] = gm == -INFINITY ? 0.f : fast_exp2(m[h] - gm);
        }
        for (int k = 0; k < Shape::kKeyGroups; ++k) {
          if (k > 0) named_bar_sync(1, kConsumerThreads);
          if (k != kg) continue;
#pragma unroll
          for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float2* dst = reinterpret_cast<float2*>(
                  merge + (rt * 16 + gid + 8 * h) * Shape::kPitch + n * 8 + 2 * tig);
              float2 x = k == 0 ? make_float2(0.f, 0.f) : *dst;
              x.x = fmaf(o[n][2 * h], f[h], x.x);
              x.y = fmaf(o[n][2 * h + 1], f[h], x.y);
              *dst = x;
            }
        }
      }
      named_bar_sync(1, kConsumerThreads);
      const bool all = end == u.begin + u.tiles && end - u.tiles >= w0;
      // A partial: slot 2c when the unit began before this CTA, else 2c + 1.
      float* part = a.part + (2 * static_cast<int64_t>(blockIdx.x) + (u.begin >= w0 ? 1 : 0)) *
                                 RT * (D + 2);
      for (int e = threadIdx.x; e < rows * (D / 4); e += kConsumerThreads) {
        const int r = e / (D / 4), c = e % (D / 4);
        float gm = -INFINITY, gl = 0.f;
#pragma unroll
        for (int k = 0; k < Shape::kKeyGroups; ++k) gm = fmaxf(gm, s_ml[k][r][0]);
        const float b = gm == -INFINITY ? 0.f : gm;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < Shape::kKeyGroups; ++k) {
          const float w = fast_exp2(s_ml[k][r][0] - b);
          gl = fmaf(w, s_ml[k][r][1], gl);
          if (at_once) {
            const float4 y = *reinterpret_cast<const float4*>(
                merge + (k * rows + r) * Shape::kPitch + c * 4);
            x.x = fmaf(w, y.x, x.x);
            x.y = fmaf(w, y.y, x.y);
            x.z = fmaf(w, y.z, x.z);
            x.w = fmaf(w, y.w, x.w);
          }
        }
        if (!at_once) x = *reinterpret_cast<const float4*>(merge + r * Shape::kPitch + c * 4);
        if (all) {
          const float inv = inv_or_zero(gl);
          const float y[4] = {x.x * inv, x.y * inv, x.z * inv, x.w * inv};
          const int i = (row0 + r) / g, hd = (row0 + r) - i * g;
          const int64_t to = base + static_cast<int64_t>(i) * a.q_heads + hd;
          store4(static_cast<T*>(a.o) + to * D + c * 4, y);
          if (a.lse != nullptr && c == 0) a.lse[to] = row_lse(gm, gl);
        } else {
          *reinterpret_cast<float4*>(part + r * D + c * 4) = x;
          if (c == 0) *reinterpret_cast<float2*>(part + RT * D + 2 * r) = make_float2(gm, gl);
        }
      }
      if (at < w1) next_unit(p.w, a.kv_len, u);
    }
  }
}

// Join: the CTAs (c, .) merge the rows of the unit that starts inside CTA c's
// range and ends behind it, from slot 2c + 1 and the slots 2(c + 1), ... of
// the CTAs that hold the unit's other tiles.  Latency-bound (a row is two to
// some tens of partials of d floats): as many of the eight warps share a row
// as leave each about four partials, whose loads fly together; the lanes read
// all maxima at once, and the warps of a row add up in their order.  Its
// registers are bounded so that its CTAs fit beside the split kernel's and
// have found their unit when that kernel ends.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 6)
    paged_join_kernel(PagedParams p, int ctas, int RT) {
  __shared__ float4 s_o[kWarps][D / 4];
  __shared__ float s_l[kWarps], s_m[kWarps];
  const PagedArgs& a = p.a;
  const int g = a.q_heads / a.kv_heads;
  const WorkSplit split(work_total(p.w, a.kv_len), ctas);
  const int c0 = blockIdx.x;
  const int64_t w0 = split.begin(c0), w1 = split.begin(c0 + 1);
  const bool any = w0 < w1;
  const WorkUnit u = find_unit(p.w, a.kv_len, any ? w1 - 1 : 0);
  const int64_t end = u.begin + u.tiles;
  const bool joins = any && u.begin >= w0 && end > w1;
  // This grid's end is all that the stream's next operation waits for, so it has
  // to imply the split kernel's end, with nothing to join too: the first CTA of
  // every range waits whatever it finds.  (All of them waiting, the rest held up
  // the joining CTAs behind them: 84.4 -> 85.6 us for one context of 131072 keys,
  // 13.8 -> 15.4 for a short one.)
  if (joins || blockIdx.y == 0) wait_for_primary();
  if (!joins) return;
  const int n = split.owner(end - 1) - c0 + 1;  // CTAs with tiles of the unit
  const int share = n <= 4 ? 1 : n <= 8 ? 2 : n <= 16 ? 4 : 8;  // warps per row
  const int at_once = kWarps / share;                           // rows per pass
  const int row0 = (u.unit % p.row_blocks) * RT;
  const int rows = min(RT, g * a.n_new - row0);
  const int64_t stride = static_cast<int64_t>(RT) * (D + 2);
  const float* first = a.part + (2 * static_cast<int64_t>(c0) + 1) * stride;
  const auto slot = [&](int i) { return first + (i == 0 ? 0 : (2 * i - 1) * stride); };
  const int kvh = u.unit / p.row_blocks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int r0 = blockIdx.y * at_once; r0 < rows; r0 += gridDim.y * at_once) {
    const int row = r0 + warp / share;
    constexpr int V = 128 / D;  // partials a warp reads at once (16 bytes a lane)
    if (row < rows) {
      float m = -INFINITY;
      for (int i = lane; i < n; i += 32) m = fmaxf(m, slot(i)[RT * D + 2 * row]);
      m = warp_max(m);
      const float base = m == -INFINITY ? 0.f : m;
      float l = 0.f, f[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int i = (warp % share) * V + lane / (D / 4); i < n; i += share * V) {
        const float* s = slot(i);
        const float2 y = *reinterpret_cast<const float2*>(s + RT * D + 2 * row);
        const float4 x = *reinterpret_cast<const float4*>(s + row * D + lane % (D / 4) * 4);
        const float w = fast_exp2(y.x - base);
        l = fmaf(w, y.y, l);
        f[0] = fmaf(w, x.x, f[0]);
        f[1] = fmaf(w, x.y, f[1]);
        f[2] = fmaf(w, x.z, f[2]);
        f[3] = fmaf(w, x.w, f[3]);
      }
      if (D == 64) {
        l += __shfl_xor_sync(0xffffffffu, l, 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] += __shfl_xor_sync(0xffffffffu, f[e], 16);
      }
      if (lane < D / 4) s_o[warp][lane] = make_float4(f[0], f[1], f[2], f[3]);
      if (lane == 0) {
        s_l[warp] = l;
        s_m[warp] = m;
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < at_once * (D / 4); e += kThreads) {
      const int k = e / (D / 4), c = e % (D / 4), r = r0 + k;
      if (r >= rows) break;
      float sum = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
      for (int i = k * share; i < (k + 1) * share; ++i) {
        sum += s_l[i];
        const float4 y = s_o[i][c];
        x[0] += y.x;
        x[1] += y.y;
        x[2] += y.z;
        x[3] += y.w;
      }
      const float inv = inv_or_zero(sum);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] *= inv;
      const int64_t at = (static_cast<int64_t>(u.seq) * a.n_new + (row0 + r) / g) * a.q_heads +
                         kvh * g + (row0 + r) % g;
      store4(static_cast<T*>(a.o) + at * D + c * 4, x);
      if (a.lse != nullptr && c == 0) a.lse[at] = row_lse(s_m[k * share], sum);
    }
    __syncthreads();
  }
}

template <typename T, int D, int R, bool CAP, bool BIAS>
cudaError_t launch_tc(const PagedTcParams& p, const PagedPlan& plan, cudaStream_t stream) {
  using Shape = PagedShape<T, D, R>;
  const cudaError_t e = ensure_max_smem<paged_tc_kernel<T, D, R, CAP, BIAS>>();
  if (e != cudaSuccess) return e;
  paged_tc_kernel<T, D, R, CAP, BIAS><<<plan.ctas, Shape::kThreadCount, Shape::kSmem, stream>>>(p);
  return cudaGetLastError();
}

template <typename T, int D, int R>
cudaError_t launch_tc_opts(const PagedTcParams& p, const PagedPlan& plan, cudaStream_t stream) {
  const bool bias = p.p.o.slopes != nullptr;
  if (p.p.o.cap > 0.f)
    return bias ? launch_tc<T, D, R, true, true>(p, plan, stream)
                : launch_tc<T, D, R, true, false>(p, plan, stream);
  return bias ? launch_tc<T, D, R, false, true>(p, plan, stream)
              : launch_tc<T, D, R, false, false>(p, plan, stream);
}

template <typename T, int D>
cudaError_t launch_tc_rows(const PagedArgs& a, const PagedPlan& plan, cudaStream_t stream) {
  PagedTcParams p;
  p.p = paged_params(a, plan);
  p.box_rows = std::min(a.page_size, KT);
  p.page_shift = 0;
  while ((1 << p.page_shift) < a.page_size) ++p.page_shift;
  p.inject_polls = consume_wait_injection();
  const cuuint64_t dims[2] = {D, static_cast<cuuint64_t>(a.n_pages) * a.kv_heads * a.page_size};
  const cuuint64_t strides[1] = {D * sizeof(T)};
  const cuuint32_t box[2] = {128 / sizeof(T), static_cast<cuuint32_t>(p.box_rows)};
  const CUtensorMapDataType type =
      sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (!encode_tile_map(&p.tk, type, a.k_pages, 2, dims, strides, box) ||
      !encode_tile_map(&p.tv, type, a.v_pages, 2, dims, strides, box))
    return cudaErrorInvalidValue;
  if (plan.row_block == 16) return launch_tc_opts<T, D, 1>(p, plan, stream);
  if (plan.row_block == 32) return launch_tc_opts<T, D, 2>(p, plan, stream);
  return launch_tc_opts<T, D, 4>(p, plan, stream);
}

// The join starts while the split kernel still runs (programmatic dependent
// launch) and waits for its partials in the kernel.
template <typename T, int D>
cudaError_t launch_join(const PagedArgs& a, const PagedPlan& plan, cudaStream_t stream) {
  const int rows = std::min(plan.row_block, a.q_heads / a.kv_heads * a.n_new);
  cudaLaunchConfig_t cfg = {};
  // About eight CTAs an SM in all; each loops over its share of the rows.
  cfg.gridDim = dim3(plan.ctas, std::max(1, std::min(rows, 8 * device_sm_count() / plan.ctas)));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<T, D>, paged_params(a, plan), plan.ctas,
                            plan.row_block);
}

}  // namespace

PagedPlan plan_paged(const PagedArgs& a, int sm_count) {
  PagedPlan p;
  const int rows = a.q_heads / a.kv_heads * a.n_new;
  p.row_block = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
  const int64_t units = static_cast<int64_t>(a.n_seqs) * a.kv_heads *
                        ((rows + p.row_block - 1) / p.row_block);
  const int64_t tiles =
      units * ((static_cast<int64_t>(a.table_pages) * a.page_size + KT - 1) / KT);
  const int per_sm = p.row_block == 16 && a.dtype == WF_BF16 ? 2 : 1;
  p.ctas = static_cast<int>(std::min<int64_t>(sm_count * per_sm, tiles));
  p.part_bytes = static_cast<size_t>(p.ctas) * 2 * p.row_block * (a.head_dim + 2) * sizeof(float);
  return p;
}

namespace {
template <typename T, int D>
cudaError_t launch_paged(const PagedArgs& a, const PagedPlan& plan, cudaStream_t stream) {
  const cudaError_t e = launch_tc_rows<T, D>(a, plan, stream);
  return e != cudaSuccess ? e : launch_join<T, D>(a, plan, stream);
}
}  // namespace

cudaError_t launch_paged_attn(const PagedArgs& a, const PagedPlan& plan, cudaStream_t stream) {
  if (a.dtype == WF_F32)
    return a.head_dim == 128 ? launch_paged<float, 128>(a, plan, stream)
                             : launch_paged<float, 64>(a, plan, stream);
  return a.head_dim == 128 ? launch_paged<__nv_bfloat16, 128>(a, plan, stream)
                           : launch_paged<__nv_bfloat16, 64>(a, plan, stream);
}

}  // namespace wf
