// Attention over packed sequences (bf16) on the fifth-generation tensor
// cores: eq. (1) per sequence, O = softmax(scale Q Kᵀ) V with the masks,
// cap and bias of wf_attn.cuh.  fp32 inputs run on the FMA pipes
// (wf_attn_fma.cu).
//
// A CTA owns two 128-row query tiles that share their keys: two query heads
// of one key-value head where the group is even (same rows, same masks, no
// half-empty pair in short sequences), else two consecutive row blocks of
// one head.  Warps 0-3 and 4-7 are the softmax groups of the two
// tiles (one thread a query row), warp 8 issues every tcgen05.mma, warp 9
// every tensor copy.  Per 128-key tile j and query tile t
//     S_t = Q_t K_jᵀ              (tcgen05, both operands in shared memory)
//     P_t = 2^(z - m)             (softmax group: registers, P over S's columns)
//     O_t += P_t V_j              (tcgen05, P from tensor memory, V row-major)
// issued as PV_0(j) QK_0(j+1) PV_1(j) QK_1(j+1): while one group works on its
// scores the tensor cores run the other tile's products.  Tensor memory:
// S_0 S_1 O_0 O_1 (512 columns of fp32 at d = 128); keys and values pass
// through one ring of 128-row stages (tensor copies, 128-byte swizzle).
//
// Visible keys of a row are always a prefix [0, limit) of its sequence
// (limit = max(position + 1, prefix) under the causal mask), so a mask is one
// comparison, only on tiles that cross some limit, and tiles behind every
// limit are never loaded.  The running maximum is only raised when a score
// exceeds it by more than 2^8 (then O is rescaled in tensor memory): the
// weights stay below 2^8, which costs no accuracy in fp32 or bf16, and after
// the first tiles O is hardly ever touched.  Weights are rounded to bf16 for
// the product with the values (half a step, 2^-8 relative each, as any bf16
// operand); their sum is taken in fp32 before that rounding.
//
// Rows behind the sequence's last key in a stage (another sequence's, or the
// copy's zero fill) meet weights of exactly 0: the softmax group clears up to
// 15 value rows there, and the product stops at the next multiple of 16.
#include <algorithm>

#include "wf_attn.cuh"
#include "wf_tensormap.h"
#include "wf_umma.cuh"

namespace wf {

namespace {

// Three warpgroups: two softmax groups and the one that issues products and
// copies (its other two warps idle).  Launched with 168 registers a thread,
// of which the issuing group hands over what the softmax groups need to keep
// a row's 128 scores in registers (8 warps x 208 + 4 x 80 <= 12 x 168).
constexpr int kPreThreads = 384;
constexpr int kIssueRegs = 80, kSoftmaxRegs = 208;
static_assert(8 * kSoftmaxRegs + 4 * kIssueRegs <= 12 * 168, "beyond the launch's registers");
constexpr int kTileRows = 128;  // query rows of a tile, keys of a tile
constexpr float kLazy = 8.f;    // log2 growth of a maximum that is tolerated

template <int D>
struct PreShape {
  static constexpr int kTileBytes = kTileRows * D * 2;
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr size_t kSmem = 1024 + (2 + kStages) * static_cast<size_t>(kTileBytes);
};

struct PrefillTcParams {
  CUtensorMap tq, tk, tv;
  PrefillArgs a;
  ScoreOpts o;
  int pair_heads;  // 1: tiles are heads h, h + 1; 0: row blocks 2b, 2b + 1
};

struct PreBarriers {
  uint64_t full[8], empty[8], q[2], s[2], p[2], o[2], drain;
  uint32_t tmem;
  int abort;
};

// A bounded wait that also ends when another role has given up.
__device__ __forceinline__ bool pre_wait(PreBarriers& b, uint64_t* bar, uint32_t parity,
                                         int32_t* status) {
  for (uint32_t i = 0; i < kWaitPolls; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 255) == 255 && *reinterpret_cast<volatile int*>(&b.abort) != 0) return false;
  }
  raise_flag(status, WF_DEV_WAIT_TIMEOUT);
  *reinterpret_cast<volatile int*>(&b.abort) = 1;
  return false;
}

__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, int x, int y, int z,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

#define WF_O8(a, i)                                                                      \
  "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3]), "=r"(a[i + 4]), "=r"(a[i + 5]), \
      "=r"(a[i + 6]), "=r"(a[i + 7])
#define WF_I8(a, i)                                                                  \
  "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3]), "r"(a[i + 4]), "r"(a[i + 5]), \
      "r"(a[i + 6]), "r"(a[i + 7])

// 64 (or 32) columns of this thread's tensor-memory lane.  The load and its
// wait are one statement: the registers of an asynchronous load must not be
// touched, moved or spilled before it.
__device__ __forceinline__ void tmem_ld64(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
      "%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,"
      "%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : WF_O8(r, 0), WF_O8(r, 8), WF_O8(r, 16), WF_O8(r, 24), WF_O8(r, 32), WF_O8(r, 40),
        WF_O8(r, 48), WF_O8(r, 56)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
      "%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : WF_O8(r, 0), WF_O8(r, 8), WF_O8(r, 16), WF_O8(r, 24)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
      "%24,%25,%26,%27,%28,%29,%30,%31};" ::WF_I8(r, 0),
      WF_I8(r, 8), WF_I8(r, 16), WF_I8(r, 24), "r"(addr)
      : "memory");
}
#undef WF_O8
#undef WF_I8
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// D[tmem] (+)= A * B with A (bf16, K packed two to a column) in tensor memory.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Row-major values as the B operand of P V (N = d contiguous): 128-byte
// swizzled, 64-column blocks `block` bytes apart (leading offset), 8-row
// groups 1024 bytes apart (stride offset).
__device__ __forceinline__ uint64_t umma_desc_rows(uint32_t saddr, uint32_t block) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) |
         (static_cast<uint64_t>((block >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// z = [cap tanh(s / cap) or scale s] - slope |d0 - i|, in the log2 domain,
// for the keys i = 0..31 of a chunk; d0 = position minus the chunk's first
// key.  `side`: every row of the warp lies behind the chunk (1: the distance
// is linear in i), before it (-1), or neither (0).
//
// cap tanh(x) = cap - 2 cap / (1 + e^(2x)).  The special-function unit is what
// bounds these variants (two powers of two and a reciprocal a score), so two
// scores share one reciprocal: 1/a = b / (a b).  With 2x log2 e clamped at 60
// the product stays finite, and 2 / (1 + 2^60) is far below fp32's step at 1.
template <bool CAP, bool BIAS>
__device__ __forceinline__ void map_scores(float* s, const ScoreOpts& o, float slope, float d0,
                                           int side) {
  const float step = side > 0 ? slope : -slope;
  const float base = (CAP ? o.cap : 0.f) - (BIAS ? step * d0 : 0.f);
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    float add[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (!BIAS)
        add[e] = base;
      else if (side != 0)
        add[e] = fmaf(step, static_cast<float>(i + e), base);
      else
        add[e] = fmaf(-slope, fabsf(d0 - static_cast<float>(i + e)), CAP ? o.cap : 0.f);
    }
    if (CAP) {
      const float k = o.scale * (2.f * kLog2e);
      const float a = 1.f + fast_exp2(fminf(s[i] * k, 60.f));
      const float b = 1.f + fast_exp2(fminf(s[i + 1] * k, 60.f));
      float r;
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a * b));
      r *= -2.f * o.cap;
      s[i] = fmaf(r, b, add[0]);
      s[i + 1] = fmaf(r, a, add[1]);
    } else {
      s[i] = fmaf(s[i], o.scale, add[0]);
      s[i + 1] = fmaf(s[i + 1], o.scale, add[1]);
    }
  }
}

// What a query tile of this CTA covers.
struct QueryTile {
  int head, row0, rows;  // head, first row within the sequence, rows (0: none)
  int end;               // keys some row sees
  int tiles;             // key tiles
};

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kPreThreads, 1)
    prefill_tc_kernel(const __grid_constant__ PrefillTcParams p) {
  using Shape = PreShape<D>;
  constexpr int kStages = Shape::kStages, kTileBytes = Shape::kTileBytes;
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) PreBarriers bars;
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  unsigned char* ring = smem + 2 * kTileBytes;
  const PrefillArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (blockIdx.x == 0) {
    check_offsets(a.cu_q, a.n_docs, a.rows_q, a.status);
    check_offsets(a.cu_k, a.n_docs, a.rows_k, a.status);
  }
  // The item: heads run fastest, a sequence's row blocks from its last (the
  // longest under the causal mask) to its first.
  const int heads = p.pair_heads ? a.q_heads / 2 : a.q_heads;
  const int block_rows = p.pair_heads ? kTileRows : 2 * kTileRows;
  DocBlock doc;
  if (!find_doc_block(a, blockIdx.x / heads, block_rows, 1, &doc)) return;
  const int hx = blockIdx.x % heads;
  doc.block = (doc.n_q + block_rows - 1) / block_rows - 1 - doc.block;
  const int prefix = p.o.prefix != nullptr ? __ldg(p.o.prefix + doc.doc) : 0;
  const int shift = doc.n_k - doc.n_q;  // position of row 0
  QueryTile qt[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    qt[t].head = p.pair_heads ? 2 * hx + t : hx;
    qt[t].row0 = doc.block * block_rows + (p.pair_heads ? 0 : t * kTileRows);
    qt[t].rows = max(0, min(kTileRows, doc.n_q - qt[t].row0));
    qt[t].end = qt[t].rows == 0 ? 0
                                : max(0, visible_end(doc.n_k, shift + qt[t].row0 + qt[t].rows - 1,
                                                     p.o.causal, prefix));
    qt[t].tiles = (qt[t].end + kTileRows - 1) / kTileRows;
  }
  const int tiles = max(qt[0].tiles, qt[1].tiles);
  const int kvh = qt[0].head / (a.q_heads / a.kv_heads);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars.q[t], 1);
      mbar_init(&bars.s[t], 1);
      mbar_init(&bars.p[t], 128);
      mbar_init(&bars.o[t], 1);
    }
    mbar_init(&bars.drain, 1);
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == 8) tmem_alloc(&bars.tmem, 512);
  if (warp == 9 && lane == 0) {
    prefetch_tensormap(&p.tq);
    prefetch_tensormap(&p.tk);
    prefetch_tensormap(&p.tv);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;
  const uint32_t tS[2] = {tmem, tmem + 128};
  const uint32_t tO[2] = {tmem + 256, tmem + 256 + D};

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == 9) {
      if (lane == 0) {
        bool ok = true;
        int fills = 0;
        for (int t = 0; t < 2; ++t) {
          if (qt[t].tiles == 0) continue;
          mbar_arrive_expect_tx(&bars.q[t], kTileBytes);
          for (int kb = 0; kb < D / 64; ++kb)
            tma_load_3d(smem + t * kTileBytes + kb * (kTileRows * 128), &p.tq, kb * 64, qt[t].head,
                        static_cast<int>(doc.q0) + qt[t].row0, &bars.q[t]);
        }
        for (int f = 0; f < 2 * tiles && ok; ++f) {
          const int st = f % kStages;
          if (f >= kStages) {
            ok = pre_wait(bars, &bars.empty[st], (f / kStages - 1) & 1, a.status);
            if (!ok) break;
          }
          unsigned char* dst = ring + st * kTileBytes;
          mbar_arrive_expect_tx(&bars.full[st], kTileBytes);
          for (int kb = 0; kb < D / 64; ++kb)
            tma_load_3d(dst + kb * (kTileRows * 128), (f & 1) ? &p.tv : &p.tk, kb * 64, kvh,
                        static_cast<int>(doc.k0) + (f >> 1) * kTileRows, &bars.full[st]);
          fills = f + 1;
        }
        if (!ok) {  // nothing of this CTA's copies may land after it has gone
          for (int t = 0; t < 2; ++t)
            if (qt[t].tiles != 0) mbar_wait_bounded(&bars.q[t], 0, a.status);
          for (int f = max(0, fills - kStages); f < fills; ++f)
            mbar_wait_bounded(&bars.full[f % kStages], (f / kStages) & 1, a.status);
        }
      }
    } else if (warp == 8) {
      // The whole warp walks the loop (uniform addresses and descriptors), one
      // elected lane issues.
      const bool leader = elect_one();
      bool ok = true;
      constexpr uint32_t kRowDesc = umma_idesc_bf16(kTileRows, D) | (1u << 16);  // B: N-major
      const uint64_t q_desc[2] = {umma_desc_sw128(smem_u32(smem)),
                                  umma_desc_sw128(smem_u32(smem + kTileBytes))};
      const uint64_t k_desc = umma_desc_sw128(smem_u32(ring));
      const uint64_t v_desc = umma_desc_rows(smem_u32(ring), kTileRows * 128);
      // S_t = Q_t K_jᵀ over the keys some row sees, rounded up to 16.
      const auto issue_qk = [&](int t, int j, int st) {
        const int n = min(kTileRows, (qt[t].end - j * kTileRows + 15) & ~15);
        const uint32_t idesc = umma_idesc_bf16(kTileRows, n);
        const uint64_t kd = k_desc + static_cast<uint32_t>(st * (kTileBytes >> 4));
        if (leader) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            constexpr int kBlock = kTileRows * 128;
            const uint32_t off = ((ks >> 2) * kBlock + (ks & 3) * 32) >> 4;
            umma_bf16(tS[t], q_desc[t] + off, kd + off, idesc, ks != 0);
          }
          umma_commit(&bars.s[t]);
        }
      };
      const auto issue_pv = [&](int t, int j, int st) {
        const int steps = min(kTileRows, qt[t].end - j * kTileRows + 15) / 16;
        const uint64_t vd = v_desc + static_cast<uint32_t>(st * (kTileBytes >> 4));
        if (leader) {
          if (steps == 8) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              umma_bf16_ts(tO[t], tS[t] + ks * 8, vd + ks * (2048 >> 4), kRowDesc, (j | ks) != 0);
          } else {
            for (int ks = 0; ks < steps; ++ks)
              umma_bf16_ts(tO[t], tS[t] + ks * 8, vd + ks * (2048 >> 4), kRowDesc, (j | ks) != 0);
          }
          if (j + 1 == qt[t].tiles) umma_commit(&bars.o[t]);
        }
      };
      const auto release = [&](int st) {
        if (leader) umma_commit(&bars.empty[st]);
      };
      // Stage and parity of the ring's fills in order: K_0 V_0 K_1 V_1 ...
      int st = 0;
      uint32_t parity = 0;
      const auto advance = [&]() {
        if (++st == kStages) {
          st = 0;
          parity ^= 1;
        }
      };
      if (tiles > 0) {
        ok = pre_wait(bars, &bars.full[0], 0, a.status);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (qt[t].tiles == 0 || !ok) continue;
          ok = pre_wait(bars, &bars.q[t], 0, a.status);
          if (ok) issue_qk(t, 0, 0);
        }
        if (ok) release(0);
        advance();
      }
      for (int j = 0; j < tiles && ok; ++j) {
        const int vs = st;
        ok = pre_wait(bars, &bars.full[vs], parity, a.status);
        advance();
        const int ks = st;
        const uint32_t kpar = parity;
        const bool more = j + 1 < tiles;
        if (more) advance();
        bool key_ready = false;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (j >= qt[t].tiles || !ok) continue;
          ok = pre_wait(bars, &bars.p[t], j & 1, a.status);
          if (!ok) continue;
          tc_fence_after();
          issue_pv(t, j, vs);
          if (j + 1 < qt[t].tiles) {
            if (!key_ready) ok = pre_wait(bars, &bars.full[ks], kpar, a.status);
            key_ready = true;
            if (ok) issue_qk(t, j + 1, ks);
          }
        }
        if (ok) {
          release(vs);
          if (more) release(ks);
        }
      }
      if (!ok) {  // the products in flight end before tensor memory is freed
        if (leader) {
          umma_commit(&bars.drain);
          mbar_wait_bounded(&bars.drain, 0, a.status);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int t = warp >> 2;
    const QueryTile me = t == 0 ? qt[0] : qt[1];
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_addr = (t == 0 ? tS[0] : tS[1]) + lanes;
    const uint32_t o_addr = (t == 0 ? tO[0] : tO[1]) + lanes;
    const int pos = shift + me.row0 + row;
    const int limit = row < me.rows
                          ? (p.o.causal ? min(doc.n_k, max(pos + 1, prefix)) : doc.n_k)
                          : me.end;
    const float slope = BIAS ? __ldg(p.o.slopes + me.head) * kLog2e : 0.f;
    // Scores (with cap or bias: mapped scores) enter the exponent as
    // fma(s, mul, -m).
    const float mul = CAP || BIAS ? 1.f : p.o.scale;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < me.tiles; ++j) {
      ok = pre_wait(bars, &bars.s[t], j & 1, a.status);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const int k0 = j * kTileRows;
      uint32_t sr[128];
      tmem_ld64(s_addr, sr);
      tmem_ld64(s_addr + 64, sr + 64);
      float* s = reinterpret_cast<float*>(sr);
      if (CAP || BIAS) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float d0 = static_cast<float>(pos - k0 - 32 * c);
          const int side = !BIAS ? 1
                           : __all_sync(0xffffffffu, d0 >= 31.f) ? 1
                           : __all_sync(0xffffffffu, d0 <= 0.f)  ? -1 : 0;
          map_scores<CAP, BIAS>(s + 32 * c, p.o, slope, d0, side);
        }
      }
      const int rel = limit - k0;
      if (__any_sync(0xffffffffu, rel < 128)) {
#pragma unroll
        for (int i = 0; i < 128; ++i) s[i] = i < rel ? s[i] : -INFINITY;
      }
      float mx0 = s[0], mx1 = s[1], mx2 = s[2], mx3 = s[3];
#pragma unroll
      for (int i = 4; i < 128; i += 4) {
        mx0 = fmaxf(mx0, s[i]);
        mx1 = fmaxf(mx1, s[i + 1]);
        mx2 = fmaxf(mx2, s[i + 2]);
        mx3 = fmaxf(mx3, s[i + 3]);
      }
      const float mt = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * mul;
      if (j == 0) {
        m = mt;
      } else if (__any_sync(0xffffffffu, mt > m + kLazy)) {
        const float mn = fmaxf(m, mt);
        const float f = mn == -INFINITY ? 1.f : fast_exp2(m - mn);
        m = mn;
        l *= f;
        const uint64_t f2 = pack2(f, f);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(o_addr + 32 * c, o);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float x, y;
            unpack2(mul2(pack2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), f2), x, y);
            o[i] = __float_as_uint(x);
            o[i + 1] = __float_as_uint(y);
          }
          tmem_st32(o_addr + 32 * c, o);
        }
      }
      const float base = m == -INFINITY ? 0.f : m;
      const uint64_t mul2v = pack2(mul, mul), base2 = pack2(-base, -base);
      uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t pk[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const int e = 64 * c + 2 * i;
          float x, y;
          unpack2(fma2(pack2(s[e], s[e + 1]), mul2v, base2), x, y);
          x = fast_exp2(x);
          y = fast_exp2(y);
          if (i & 1) sum1 = add2(sum1, pack2(x, y)); else sum0 = add2(sum0, pack2(x, y));
          const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
          pk[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        tmem_st32(s_addr + 32 * c, pk);
      }
      float a0, a1;
      unpack2(add2(sum0, sum1), a0, a1);
      l += a0 + a1;
      // Value rows behind the last key of the sequence, up to the product's end.
      if (doc.n_k - k0 < kTileRows) {
        const int r0 = doc.n_k - k0, r1 = min(kTileRows, (me.end - k0 + 15) & ~15);
        if (r0 < r1) {
          const int f = 2 * j + 1;
          ok = pre_wait(bars, &bars.full[f % kStages], (f / kStages) & 1, a.status);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          unsigned char* v = ring + (f % kStages) * kTileBytes;
          for (int e = row; e < (r1 - r0) * (D / 8); e += 128) {
            const int r = r0 + e / (D / 8), c = e % (D / 8);
            *reinterpret_cast<uint4*>(v + (c >> 3) * (kTileRows * 128) + r * 128 + (c & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async();
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&bars.p[t]);
    }
    if (ok && me.tiles > 0) {
      ok = pre_wait(bars, &bars.o[t], 0, a.status);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
    }
    if (ok) {
      const float inv = inv_or_zero(l);
      const bool live = row < me.rows;
      const int64_t at = (doc.q0 + me.row0 + row) * a.q_heads + me.head;
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.o) + at * D;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (me.tiles > 0) {
          tmem_ld32(o_addr + 32 * c, o);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0;
        }
        if (live) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              // A row without a visible key: nothing was summed, 0 whatever O holds.
              const float x = l == 0.f ? 0.f : __uint_as_float(o[i + 2 * e]) * inv;
              const float y = l == 0.f ? 0.f : __uint_as_float(o[i + 2 * e + 1]) * inv;
              const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
              w[e] = *reinterpret_cast<const uint32_t*>(&b);
            }
            *reinterpret_cast<uint4*>(dst + 32 * c + i) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (live && a.lse != nullptr) a.lse[at] = row_lse(m, l);
    }
  }
  __syncwarp();  // the issuing lanes rejoin their warps
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

// [rows, heads, d] bf16 with a row stride, boxes of 64 columns x 1 head x 128
// rows, 128-byte swizzle; rows outside read as zero.
bool encode_rows(CUtensorMap* map, const void* base, int64_t rows, int heads, int d,
                 int64_t stride) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2,
                                 static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[3] = {64, 1, kTileRows};
  return encode_bf16_map(map, base, 3, dims, strides, box);
}

template <int D, bool CAP, bool BIAS>
cudaError_t launch_tc(const PrefillTcParams& p, cudaStream_t stream) {
  const cudaError_t e = ensure_max_smem<prefill_tc_kernel<D, CAP, BIAS>>();
  if (e != cudaSuccess) return e;
  const int block_rows = p.pair_heads ? kTileRows : 2 * kTileRows;
  const int64_t items = doc_blocks(p.a.rows_q, p.a.n_docs, block_rows, 1) *
                        (p.pair_heads ? p.a.q_heads / 2 : p.a.q_heads);
  if (items > INT32_MAX) return cudaErrorInvalidValue;
  prefill_tc_kernel<D, CAP, BIAS>
      <<<static_cast<unsigned>(items), kPreThreads, PreShape<D>::kSmem, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_tc_opts(const PrefillTcParams& p, cudaStream_t stream) {
  const bool bias = p.o.slopes != nullptr;
  if (p.o.cap > 0.f)
    return bias ? launch_tc<D, true, true>(p, stream) : launch_tc<D, true, false>(p, stream);
  return bias ? launch_tc<D, false, true>(p, stream) : launch_tc<D, false, false>(p, stream);
}

}  // namespace

cudaError_t launch_prefill(const PrefillArgs& a, cudaStream_t stream) {
  if (a.dtype == WF_F32) return launch_prefill_fma(a, stream);
  PrefillTcParams p;
  p.a = a;
  p.o = score_opts(a.scale, a.softcap, a.causal, a.prefix, a.slopes);
  p.pair_heads = (a.q_heads / a.kv_heads) % 2 == 0;
  // Without keys no copy of them is ever issued; the maps only have to exist.
  const bool keys = a.rows_k > 0;
  if (!encode_rows(&p.tq, a.q, a.rows_q, a.q_heads, a.head_dim, a.q_stride) ||
      !encode_rows(&p.tk, keys ? a.k : a.q, keys ? a.rows_k : 1, a.kv_heads, a.head_dim,
                   a.k_stride) ||
      !encode_rows(&p.tv, keys ? a.v : a.q, keys ? a.rows_k : 1, a.kv_heads, a.head_dim,
                   a.v_stride))
    return cudaErrorInvalidValue;
  return a.head_dim == 128 ? launch_tc_opts<128>(p, stream) : launch_tc_opts<64>(p, stream);
}

}  // namespace wf
