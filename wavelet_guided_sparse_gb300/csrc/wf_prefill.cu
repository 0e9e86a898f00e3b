// Attention over packed sequences (bf16) on the fifth-generation tensor
// cores: eq. (1) per sequence, O = softmax(scale Q Kᵀ) V with the masks,
// cap and bias of wf_attn.cuh.  fp32 inputs run on the FMA pipes
// (wf_attn_fma.cu).
//
// An item is two 128-row query tiles that share their keys: two query heads
// of one key-value head where the group is even (same rows, same masks, no
// half-empty pair in short sequences), else two consecutive row blocks of one
// head.  Warp 0 issues every tcgen05.mma, warp 1 every tensor copy, warp 2
// finds the items (warp 3 idles); warps 4-7 and 8-11 are the softmax groups of
// the two tiles, one thread a query row.  Per 128-key tile j and query tile t
//     S_t = Q_t K_jᵀ              (both operands in shared memory)
//     P_t = 2^(z - m)             (softmax group, in place of S_t's columns)
//     O_t += P_t V_j              (P from tensor memory, V row-major)
// issued as PV_0(j) QK_0(j-1) PV_1(j) QK_1(j-1), from the last key tile to the
// first: while one group works on its scores the tensor cores run the other
// tile's products.  Tensor memory: S_0 S_1 O_0 O_1 (512 columns of fp32 at
// d = 128); keys and values pass through one ring of 128-row stages (tensor
// copies, 128-byte swizzle).
//
// Visible keys of a row are always a prefix [0, limit) of its sequence
// (limit = max(position + 1, prefix) under the causal mask), so a mask is a
// word of bits per 32 keys, only on tiles that cross some limit, and tiles
// behind every limit are never loaded.  The running maximum is set 8 (in log2)
// above the score that raises it and raised again, O rescaled in tensor memory,
// only by a score beyond that: after the first tiles O is hardly ever touched,
// and the weights stay below 1, so that a value of the type's largest does not
// overflow on the way.  Weights are
// rounded to bf16 for the product with the values (half a step, 2^-8 relative
// each, as any bf16 operand); their sum is taken in fp32 before that rounding.
//
// A CTA stays on its SM: warp 2 claims blocks of the grid that have not
// started yet (cluster launch control: dynamic balance without a counter in
// memory), one item ahead of the one in work, so that the next item's
// queries, keys and first scores come in behind the current one's last tiles
// and output.
//
// Rows behind the sequence's last key in a stage (another sequence's, or the
// copy's zero fill) meet weights of exactly 0: the softmax group clears up to
// 15 value rows there, and the product stops at the next multiple of 16.
//
// Measured (32 query heads, 8 of keys, d = 128): 8192 rows over 8192 keys 690
// us, 1593 TFLOP/s, 82 % of cuBLAS's bf16 rate; causal 362 to 368 us.  The
// softmax bounds it: a step of 128 keys for both tiles takes 2930 cycles, of
// which the products fill 2048; the exponentials, FMAs and conversions of
// 2 x 128 x 128 scores and the two hand-overs between the roles fill the
// rest.  A short sequence adds per item its first tile (2200 cycles, whose
// masks cost twice) and the output (2700): packed prompts of 20 to 3000 rows
// 194 us, 53 %.  With cap and bias the mapping of the scores (8 FMA results
// each, at 128 a cycle and SM) lies on the same chain: 616 us for 8192 causal
// rows, 2329 us (49 %) for 16384.
#include <algorithm>

#include "wf_attn.cuh"
#include "wf_tensormap.h"
#include "wf_umma.cuh"

namespace wf {

namespace {

// Three warpgroups: the issuing one and two of softmax.  Launched with 168
// registers a thread, of which the issuing group hands over what the softmax
// groups use beyond that (8 warps x 208 + 4 x 80 <= 12 x 168).
constexpr int kPreThreads = 384;
constexpr int kIssueRegs = 80, kSoftmaxRegs = 208;
static_assert(8 * kSoftmaxRegs + 4 * kIssueRegs <= 12 * 168, "beyond the launch's registers");
// Warps 0-3 issue, 4-7 and 8-11 are the softmax groups.
constexpr int kProducts = 0, kCopies = 1, kItems = 2;
constexpr int kTileRows = 128;  // query rows of a tile, keys of a tile
constexpr float kHeadroom = 8.f;  // a maximum above the score that raised it (log2)

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
  int capped;      // 1: the grid has fewer blocks than items there might be
  uint32_t inject_polls;  // fault injection (tests): see the kernel's start
};

// What a query tile of an item covers.
struct QueryTile {
  int head, row0, rows;  // head, first row within the sequence, rows (0: none)
  int end;               // keys some row sees
  int tiles;             // key tiles
};
// One unit of work: two query tiles over their sequence's keys.
struct Item {
  QueryTile qt[2];
  int q0, k0, n_k, shift, prefix;  // first row and key, keys, position of row 0
  int kvh, live;                   // key-value head; 0: no more items
};

struct PreBarriers {
  uint64_t full[8];            // ring stages
  uint64_t done[8];            // steps (below) whose stages are free again: at most
                               // five lie between a copy's wait and the products
  uint64_t q[2], q_empty[2];   // query tiles in shared memory
  uint64_t s[2], p[2];         // scores ready; weights ready
  uint64_t o[2], o_empty[2];   // output finished; read
  uint64_t item[2], item_empty[2];  // item published; read by every role
  uint64_t claim, drain;
  uint4 claimed;               // response of a claim
  Item it[2];
  uint32_t tmem;
  WaitState wait;
};

__device__ __forceinline__ bool pre_wait(PreBarriers& b, uint64_t* bar, uint32_t parity,
                                         int32_t* status, uint32_t nap = 0) {
  return warp_wait(bar, parity, b.wait, status, nap);
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

// 64 (32, 16) columns of this thread's tensor-memory lane.  The load and its
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
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : WF_O8(r, 0), WF_O8(r, 8)
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
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::WF_I8(r, 0),
      WF_I8(r, 8), "r"(addr)
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

// The smaller of two numbers, NaN if one is NaN (a visible key that holds one
// has to show in its rows).
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// What maps a query row's scores, kept over an item (pairs: both lanes of an
// f32x2 operation).
struct ScoreMap {
  uint64_t scale;        // no cap: scale log2 e
  uint64_t bend[5];      // cap: coefficients of cap log2 e tanh(s scale / cap) / s in s^2
  uint64_t steps[16];    // slope times (2 i, 2 i + 1)
  float slope;           // slope log2 e
  float weigh;           // cap: scale / cap, 0 in a row that does not exist
};

// z = [cap tanh(s / cap) or scale s] - slope |d0 - i|, in the log2 domain,
// for the keys i = 0..31 of a chunk; d0 = position minus the chunk's first
// key.  `side`: every row of the warp lies behind the chunk (1: the distance
// is linear in i), before it (-1), or neither (0).
//
// The cap: while every |s scale / cap| of the warp's chunk is at most 1/2, the
// usual case, the polynomial of tanh_exp2 on the FMA pipe, two scores an
// operation, its coefficients scaled so that it takes s itself.  Otherwise
// tanh(x) = 1 - 2 / (1 + e^(2x)) on the special-function unit, two scores
// sharing one reciprocal (1/a = b / (a b)); with 2x log2 e clamped at 60 the
// product stays finite, and 2 / (1 + 2^60) is far below fp32's step at 1.
// That branch's error is one of the cap (2^-21 of it), not of a small score.
// Caps so far from the scale that the scaled coefficients would leave fp32's
// range (at 1/sqrt(d): above 384 for d = 128, 567 for 64, and below 2e-5) take
// tanh_exp2 as it is.  Hidden scores come as 0 (they must neither choose the
// form nor share a reciprocal), and rows that do not exist (the next sequence's
// queries) have no say in it.
template <bool CAP, bool BIAS, bool LINEAR>
__device__ __forceinline__ void map_chunk(float* s, const ScoreOpts& o, const ScoreMap& c,
                                          float d0, float sg) {
  const float base = BIAS && LINEAR ? -sg * c.slope * d0 : 0.f;
  const uint64_t base2 = pack2(base, base), sign2 = pack2(sg, sg);
  const auto bias = [&](int i) {  // of keys i, i + 1
    if (LINEAR) return fma2(c.steps[i / 2], sign2, base2);
    return pack2(-c.slope * fabsf(d0 - static_cast<float>(i)),
                 -c.slope * fabsf(d0 - static_cast<float>(i + 1)));
  };
  if (!CAP) {
#pragma unroll
    for (int i = 0; i < 32; i += 2)
      unpack2(fma2(pack2(s[i], s[i + 1]), c.scale, bias(i)), s[i], s[i + 1]);
    return;
  }
  float big0 = 0.f, big1 = 0.f;
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    big0 = fmaxf(big0, fmaxf(fabsf(s[i]), fabsf(s[i + 1])));
    big1 = fmaxf(big1, fmaxf(fabsf(s[i + 2]), fabsf(s[i + 3])));
  }
  if (__all_sync(0xffffffffu, !(fmaxf(big0, big1) * c.weigh > o.bend_max))) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const uint64_t x = pack2(s[i], s[i + 1]), u = mul2(x, x);
      uint64_t q = c.bend[4];
#pragma unroll
      for (int e = 3; e >= 0; --e) q = fma2(q, u, c.bend[e]);
      unpack2(BIAS ? fma2(x, q, bias(i)) : mul2(x, q), s[i], s[i + 1]);
    }
    return;
  }
  if (o.bend_max < 0.f) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      float x = 0.f, y = 0.f;
      if (BIAS) unpack2(bias(i), x, y);
      s[i] = fmaf(o.cap, tanh_exp2(s[i] * o.scale), x);
      s[i + 1] = fmaf(o.cap, tanh_exp2(s[i + 1] * o.scale), y);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    float add0 = o.cap, add1 = o.cap;
    if (BIAS) {
      float x, y;
      unpack2(bias(i), x, y);
      add0 += x;
      add1 += y;
    }
    const float k = o.scale * (2.f * kLog2e);
    const float a = 1.f + fast_exp2(min_nan(s[i] * k, 60.f));
    const float b = 1.f + fast_exp2(min_nan(s[i + 1] * k, 60.f));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a * b));
    r *= -2.f * o.cap;
    s[i] = fmaf(r, b, add0);
    s[i + 1] = fmaf(r, a, add1);
  }
}
// One branch a chunk, none between its scores.
template <bool CAP, bool BIAS>
__device__ __forceinline__ void map_scores(float* s, const ScoreOpts& o, const ScoreMap& c,
                                           float d0, int side) {
  if (!BIAS || side != 0)
    map_chunk<CAP, BIAS, true>(s, o, c, d0, side > 0 ? 1.f : -1.f);
  else
    map_chunk<CAP, BIAS, false>(s, o, c, d0, 0.f);
}

// A chunk's keys from `n` on are hidden: their scores become `with`.  One bit a
// key: bits of a register become predicates eight at once.
__device__ __forceinline__ void hide_keys(float* s, int n, float with = -INFINITY) {
  const uint32_t seen = n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
#pragma unroll
  for (int i = 0; i < 32; ++i) s[i] = (seen & (1u << i)) != 0 ? s[i] : with;
}

template <int N>
__device__ __forceinline__ float chunk_max(const float* s) {
  float a = -INFINITY, b = -INFINITY;
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    a = fmaxf(a, fmaxf(s[i], s[i + 1]));
    b = fmaxf(b, fmaxf(s[i + 2], s[i + 3]));
  }
  return fmaxf(a, b);
}

// Weights 2^(s mul - m), packed to bf16; their sum in fp32, in two parts.
template <int N>
__device__ __forceinline__ void chunk_weights(const float* s, float mul, float m, uint32_t* pk,
                                              uint64_t& sum0, uint64_t& sum1) {
  const float base = m == -INFINITY ? 0.f : m;
  const uint64_t mul2v = pack2(mul, mul), base2 = pack2(-base, -base);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    float x, y;
    unpack2(fma2(pack2(s[2 * i], s[2 * i + 1]), mul2v, base2), x, y);
    x = fast_exp2(x);
    y = fast_exp2(y);
    if (i & 1) sum1 = add2(sum1, pack2(x, y)); else sum0 = add2(sum0, pack2(x, y));
    const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
    pk[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
}

// Rows whose new score exceeds the maximum raise it to kHeadroom above that
// score: the weight of a row's only (or outstanding) key is then 2^-8 and meets
// no rounding.  Returns the factor for what has been summed.
//
// `rounded`: the sum of weights that are in bf16 already and follow by the same
// factor.  It is a power of two and rounds them no further, with the maximum up
// to 1 lower, unless they come to less than 2^-9 of the new score's weight: a
// second rounding of theirs is then lost in that of the result.  (Powers of two
// always: relative error 0.0022 in place of 0.0021 on a 16384-token prompt with
// cap and bias, for the outstanding keys' own rounding.)
__device__ __forceinline__ float raise_max(float& m, float mt, float rounded = 0.f) {
  if (!(mt > m)) return 1.f;
  const float old = m;
  m = mt + kHeadroom;
  const float f = fast_exp2(old - m);
  if (!(rounded * f > 0x1p-17f)) return f;  // the new score's weight is 2^-8
  const float steps = ceilf(old - m);
  m = old - steps;
  return __int_as_float((127 + static_cast<int>(steps)) << 23);
}

template <int D>
__device__ __forceinline__ void scale_output(uint32_t o_addr, float f) {
  const uint64_t f2 = pack2(f, f);
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    uint32_t o[32];
    tmem_ld32(o_addr + c, o);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      float x, y;
      unpack2(mul2(pack2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), f2), x, y);
      o[i] = __float_as_uint(x);
      o[i + 1] = __float_as_uint(y);
    }
    tmem_st32(o_addr + c, o);
  }
  tmem_wait_st();
}

// Claims a block of this grid that has not started (cluster launch control):
// the 16-byte response lands at `to`, counted on `bar`.
__device__ __forceinline__ void claim_block(uint4* to, uint64_t* bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 "
      "[%0], [%1];" ::"r"(smem_u32(to)),
      "r"(smem_u32(bar))
      : "memory");
}
// The claimed block's index, or -1 when none was left.
__device__ __forceinline__ int64_t claimed_block(const uint4* from) {
  uint32_t ok, x;
  asm volatile(
      "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
      : "=r"(ok), "=r"(x)
      : "r"(smem_u32(from))
      : "memory");
  return ok ? static_cast<int64_t>(x) : -1;
}

// An item by its index: heads run fastest, a sequence's row blocks from its
// last (the longest under the causal mask) to its first.  False: behind the
// last sequence.  Whole warp.
__device__ __forceinline__ bool make_item(const PrefillTcParams& p, int64_t index,
                                          DocCursor& cursor, Item* out) {
  const PrefillArgs& a = p.a;
  Item& it = *out;
  const int heads = p.pair_heads ? a.q_heads / 2 : a.q_heads;
  const int block_rows = p.pair_heads ? kTileRows : 2 * kTileRows;
  if (index == 0) {
    check_offsets(a.cu_q, a.n_docs, a.rows_q, a.status, threadIdx.x & 31, 32);
    check_offsets(a.cu_k, a.n_docs, a.rows_k, a.status, threadIdx.x & 31, 32);
  }
  DocBlock doc;
  if (!find_doc_block(a, index / heads, block_rows, 1, cursor, &doc)) return false;
  it.live = 1;
  const int hx = static_cast<int>(index % heads);
  doc.block = (doc.n_q + block_rows - 1) / block_rows - 1 - doc.block;
  it.q0 = static_cast<int>(doc.q0);
  it.k0 = static_cast<int>(doc.k0);
  it.n_k = doc.n_k;
  it.prefix = p.o.prefix != nullptr ? __ldg(p.o.prefix + doc.doc) : 0;
  it.shift = doc.n_k - doc.n_q;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    QueryTile& q = it.qt[t];
    q.head = p.pair_heads ? 2 * hx + t : hx;
    q.row0 = doc.block * block_rows + (p.pair_heads ? 0 : t * kTileRows);
    q.rows = max(0, min(kTileRows, doc.n_q - q.row0));
    q.end = q.rows == 0 ? 0
                        : max(0, visible_end(doc.n_k, it.shift + q.row0 + q.rows - 1, p.o.causal,
                                             it.prefix));
    q.tiles = (q.end + kTileRows - 1) / kTileRows;
  }
  it.kvh = it.qt[0].head / (a.q_heads / a.kv_heads);
  return true;
}

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

  // Fault injection (tests of the bounded waits): the first CTA's first key tile
  // is never issued, and its waits give up after inject_polls polls.
  const bool inject = p.inject_polls != 0 && blockIdx.x == 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&bars.full[i], 1);
    for (int i = 0; i < 8; ++i) mbar_init(&bars.done[i], 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars.q[t], 1);
      mbar_init(&bars.q_empty[t], 1);
      mbar_init(&bars.s[t], 1);
      mbar_init(&bars.p[t], 128);
      mbar_init(&bars.o[t], 1);
      mbar_init(&bars.o_empty[t], 128);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.item[i], 1);
      mbar_init(&bars.item_empty[i], 10);
    }
    mbar_init(&bars.claim, 1);
    mbar_init(&bars.drain, 1);
    bars.wait.init(inject ? p.inject_polls : kWaitPolls);
    fence_mbar_init();
  }
  if (warp == kProducts) tmem_alloc(&bars.tmem, 512);
  if (warp == kCopies && lane == 0) {
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

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    const bool leader = elect_one();
    if (warp == kItems) {
      // ---- items: those of this CTA's own block, then of blocks of the grid not
      // started yet; `grain` to a block, 1 unless a capped grid has too few.
      bool ok = true;
      uint32_t claims = 0;
      DocCursor cursor = {0, 0};
      int64_t grain = 1, items = INT64_MAX;  // (not counted)
      if (p.capped) {
        items = p.pair_heads ? doc_total(a, kTileRows, 1) * (a.q_heads / 2)
                             : doc_total(a, 2 * kTileRows, 1) * a.q_heads;
        grain = max(grain, (items + gridDim.x - 1) / gridDim.x);
      }
      int64_t next = blockIdx.x * grain, stop = next + grain;
      for (uint32_t k = 0; ok; ++k) {
        // The item before the last one has been read by all.
        if (k > 1) ok = pre_wait(bars, &bars.item_empty[k & 1], ((k >> 1) - 1) & 1, a.status, 200);
        if (!ok) break;
        Item it = {};
        // Blocks behind the last sequence's (the grid is sized for any split
        // of the rows) are claimed and dropped.  Item 0 is looked at even if there
        // is none, for the offsets' sake.
        while (next >= stop || (next >= items && next > 0) ||
               !make_item(p, next++, cursor, &it)) {
          if (leader) {
            fence_proxy_async();
            mbar_arrive_expect_tx(&bars.claim, 16);
            claim_block(&bars.claimed, &bars.claim);
          }
          __syncwarp();
          // Not cut short: the response must have landed before the CTA may go.
          ok = mbar_wait_bounded(&bars.claim, claims++ & 1, a.status);
          const int64_t block = ok ? claimed_block(&bars.claimed) : -1;
          if (block < 0) break;
          next = block * grain;
          stop = next + grain;
        }
        if (leader) {
          bars.it[k & 1] = it;
          mbar_arrive(&bars.item[k & 1]);
        }
        __syncwarp();
        if (!it.live) break;
      }
    } else if (warp == kCopies) {
      // ---- copies
      bool ok = true;
      uint32_t used[2] = {0, 0}, fills = 0, steps = 0;
      uint32_t step_of[kStages] = {};  // the step that frees each stage
      int st = 0;
      for (uint32_t k = 0; ok; ++k) {
        ok = pre_wait(bars, &bars.item[k & 1], (k >> 1) & 1, a.status);
        if (!ok) break;
        const Item it = bars.it[k & 1];
        __syncwarp();
        if (leader) mbar_arrive(&bars.item_empty[k & 1]);
        if (!it.live) break;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (it.qt[t].tiles == 0 || !ok) continue;
          if (used[t] > 0) ok = pre_wait(bars, &bars.q_empty[t], (used[t] - 1) & 1, a.status, 100);
          if (!ok) continue;
          ++used[t];
          if (leader) {
            mbar_arrive_expect_tx(&bars.q[t], kTileBytes);
            for (int kb = 0; kb < D / 64; ++kb)
              tma_load_3d(smem + t * kTileBytes + kb * (kTileRows * 128), &p.tq, kb * 64,
                          it.qt[t].head, it.q0 + it.qt[t].row0, &bars.q[t]);
          }
        }
        const int tiles = max(it.qt[0].tiles, it.qt[1].tiles);
        for (int f = 0; f < 2 * tiles && ok; ++f) {
          if (fills >= kStages) {
            uint32_t r = 0;
#pragma unroll
            for (int i = 0; i < kStages; ++i) r = i == st ? step_of[i] : r;
            ok = pre_wait(bars, &bars.done[r & 7], (r >> 3) & 1, a.status, 100);
          }
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < kStages; ++i)
            if (i == st) step_of[i] = steps + (f > 0 ? (f - 1) >> 1 : 0);
          if (leader && !(inject && fills == 0)) {
            unsigned char* dst = ring + st * kTileBytes;
            mbar_arrive_expect_tx(&bars.full[st], kTileBytes);
            for (int kb = 0; kb < D / 64; ++kb)
              tma_load_3d(dst + kb * (kTileRows * 128), (f & 1) ? &p.tv : &p.tk, kb * 64, it.kvh,
                          it.k0 + (tiles - 1 - (f >> 1)) * kTileRows, &bars.full[st]);
          }
          ++fills;
          if (++st == kStages) st = 0;
        }
        steps += tiles;
      }
      // Nothing of this CTA's copies may land after it has gone, also where another
      // role has given up behind this warp's last wait.
      if (leader) {
        for (int t = 0; t < 2; ++t)
          if (used[t] > 0) mbar_wait_bounded(&bars.q[t], (used[t] - 1) & 1, a.status);
        for (uint32_t f = max(inject ? 1 : 0, static_cast<int>(fills) - kStages); f < fills; ++f)
          mbar_wait_bounded(&bars.full[f % kStages], (f / kStages) & 1, a.status);
      }
    } else if (warp == kProducts) {
      // ---- products: the whole warp walks the loop, one elected lane issues.
      // A step is one key tile j: each query tile's product with V_j, then its
      // scores of K_{j-1} (before an item's first step, those of its first key
      // tile).  One arrival a step frees its stages: an arrival costs the
      // issuing warp 130 cycles.
      bool ok = true;
      constexpr uint32_t kRowDesc = umma_idesc_bf16(kTileRows, D) | (1u << 16);  // B: N-major
      const uint64_t q_desc[2] = {umma_desc_sw128(smem_u32(smem)),
                                  umma_desc_sw128(smem_u32(smem + kTileBytes))};
      const uint64_t k_desc = umma_desc_sw128(smem_u32(ring));
      const uint64_t v_desc = umma_desc_rows(smem_u32(ring), kTileRows * 128);
      // S_t = Q_t K_jᵀ over the keys some row sees, rounded up to 16.
      const auto issue_qk = [&](int t, int keys, int st) {
        const int n = min(kTileRows, (keys + 15) & ~15);
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
      // O_t += P_t V_j over `steps` 16-key steps; `fresh`: the first replaces O.
      const auto issue_pv = [&](int t, int steps, int st, bool fresh) {
        const uint64_t vd = v_desc + static_cast<uint32_t>(st * (kTileBytes >> 4));
        if (leader) {
          if (steps == 8) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              umma_bf16_ts(tO[t], tS[t] + ks * 8, vd + ks * (2048 >> 4), kRowDesc,
                           !(fresh && ks == 0));
          } else {
            for (int ks = 0; ks < steps; ++ks)
              umma_bf16_ts(tO[t], tS[t] + ks * 8, vd + ks * (2048 >> 4), kRowDesc,
                           !(fresh && ks == 0));
          }
        }
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
      uint32_t used[2] = {0, 0};  // items with tiles of query tile t so far
      uint32_t np[2] = {0, 0};    // key tiles of query tile t so far
      uint32_t step = 0;          // steps so far
      for (uint32_t k = 0; ok; ++k) {
        ok = pre_wait(bars, &bars.item[k & 1], (k >> 1) & 1, a.status);
        if (!ok) break;
        const Item& it = bars.it[k & 1];
        const int live = it.live;
        const int end[2] = {it.qt[0].end, it.qt[1].end};
        const int nt[2] = {it.qt[0].tiles, it.qt[1].tiles};
        __syncwarp();
        if (leader) mbar_arrive(&bars.item_empty[k & 1]);
        if (!live) break;
        const int tiles = max(nt[0], nt[1]);
        if (tiles == 0) continue;
        // The scores of key tile j (stage st): query tile t's first ones wait
        // for its queries, its last ones release them.
        const auto scores = [&](int t, int j, int st) {
          if (j == nt[t] - 1) ok = pre_wait(bars, &bars.q[t], used[t] & 1, a.status);
          if (!ok) return;
          issue_qk(t, end[t] - j * kTileRows, st);
          if (j == 0 && leader) umma_commit(&bars.q_empty[t]);
        };
        ok = pre_wait(bars, &bars.full[st], parity, a.status);
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (ok && nt[t] == tiles) scores(t, tiles - 1, st);
        advance();
        for (int j = tiles - 1; j >= 0 && ok; --j) {
          const int vs = st;
          ok = pre_wait(bars, &bars.full[vs], parity, a.status);
          advance();
          const int ks = st;
          const uint32_t kpar = parity;
          if (j > 0) {
            advance();
            ok = ok && pre_wait(bars, &bars.full[ks], kpar, a.status);
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (ok && j < nt[t]) {
              // The last item's output must have been read.
              if (j == nt[t] - 1 && used[t] > 0)
                ok = pre_wait(bars, &bars.o_empty[t], (used[t] - 1) & 1, a.status);
              ok = ok && pre_wait(bars, &bars.p[t], np[t] & 1, a.status);
              if (!ok) continue;
              ++np[t];
              tc_fence_after();
              issue_pv(t, min(kTileRows, end[t] - j * kTileRows + 15) / 16, vs, j == nt[t] - 1);
              if (j == 0 && leader) umma_commit(&bars.o[t]);
            }
            if (ok && j > 0 && j - 1 < nt[t]) scores(t, j - 1, ks);
          }
          if (ok && leader) umma_commit(&bars.done[step & 7]);
          ++step;
        }
        used[0] += nt[0] > 0;
        used[1] += nt[1] > 0;
      }
      // Every product, and every arrival it still owes, ends before tensor
      // memory is freed and the CTA goes.
      if (leader) umma_commit(&bars.drain);
      __syncwarp();
      mbar_wait_bounded(&bars.drain, 0, a.status);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---- softmax and output of query tile t, one row a thread
    const int t = (warp >> 2) - 1;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_addr = (t == 0 ? tS[0] : tS[1]) + lanes;
    const uint32_t o_addr = (t == 0 ? tO[0] : tO[1]) + lanes;
    const float mul = p.o.scale;  // unmapped scores enter the exponent as fma(s, mul, -m)
    uint32_t ns = 0, used = 0, fill = 0;  // key tiles, items with tiles, ring fills so far
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      ok = pre_wait(bars, &bars.item[k & 1], (k >> 1) & 1, a.status);
      if (!ok) break;
      // This thread's row: its place in the output, whether it exists (a row
      // outside the arrays is never written), its visible keys.
      const Item& it = bars.it[k & 1];
      const int mine = it.qt[t].tiles, end = it.qt[t].end, n_k = it.n_k;
      const int tiles = max(it.qt[0].tiles, it.qt[1].tiles);
      const int row_at = it.qt[t].row0 + row, head = it.qt[t].head, rows = it.qt[t].rows;
      const int64_t out_row = static_cast<int64_t>(it.q0) + row_at;
      const bool sound = static_cast<uint64_t>(out_row - row) + rows <=
                             static_cast<uint64_t>(a.rows_q) &&
                         static_cast<uint32_t>(head) < static_cast<uint32_t>(a.q_heads);
      const bool live = row < rows && sound;
      const int64_t at = out_row * a.q_heads + head;
      const int pos = it.shift + row_at, live_item = it.live;
      const int limit = live ? (p.o.causal ? min(n_k, max(pos + 1, it.prefix)) : n_k) : end;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.item_empty[k & 1]);
      if (!live_item) break;
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
        map.slope = BIAS ? __ldg(p.o.slopes + max(0, min(head, a.q_heads - 1))) * kLog2e : 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          map.steps[i] = pack2(map.slope * (2 * i), map.slope * (2 * i + 1));
      }
      float m = -INFINITY, l = 0.f;
      // From the last key tile (under the causal mask the nearest keys, whose
      // scores a distance bias leaves highest) to the first.
      for (int j = mine - 1; j >= 0; --j) {
        ok = pre_wait(bars, &bars.s[t], ns & 1, a.status);
        if (!ok) break;
        ++ns;
        tc_fence_after();
        const int k0 = j * kTileRows;
        // Chunks of scores in rolled loops: with the tile unrolled the code of the
        // softmax groups would not stay in the instruction caches, and every
        // role, the products' warp first, would wait for its fetches.  A chunk's
        // weights go over columns already read.
        const int rel = limit - k0;
        const bool edge = __any_sync(0xffffffffu, rel < 128);
        uint64_t sum0 = 0, sum1 = 0;
        if constexpr (CAP || BIAS) {
          // One pass.  The weights of a chunk are formed before the test on its
          // maximum, beside the maximum's own chain of operations, and once more
          // after the rare raise.  (Two passes, as below, would carry the mapped
          // scores through tensor memory: 644 against 618 us for 8192 causal rows
          // with cap and bias.)
          if (CAP && edge) {
            // Hidden scores become 0 in place (they may be NaN, and columns without a
            // key hold what an earlier item left): beside, not in, the loop below,
            // whose code they would slow by a tenth.
#pragma unroll 1
            for (int c = 0; c < 128; c += 32) {
              uint32_t r[32];
              tmem_ld32(s_addr + c, r);
              hide_keys(reinterpret_cast<float*>(r), rel - c, 0.f);
              tmem_st32(s_addr + c, r);
            }
            tmem_wait_st();
          }
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            uint32_t r[32], pk[16];
            tmem_ld32(s_addr + c, r);
            float* s = reinterpret_cast<float*>(r);
            const float d0 = static_cast<float>(pos - k0 - c);
            const int side = !BIAS ? 1
                             : __all_sync(0xffffffffu, d0 >= 31.f) ? 1
                             : __all_sync(0xffffffffu, d0 <= 0.f)  ? -1 : 0;
            map_scores<CAP, BIAS>(s, p.o, map, d0, side);
            if (edge) hide_keys(s, rel - c);
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
              if (f != 1.f) {  // other rows' sums go on in their order
                l = (l + (a0 + a1)) * f;
                sum0 = sum1 = 0;
              }
              if (c > 0) tmem_wait_st();
              const __nv_bfloat162 fb = __float2bfloat162_rn(f);
#pragma unroll 1
              for (int e = 0; e < c / 2; e += 16) {
                uint32_t w[16];
                tmem_ld16(s_addr + e, w);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const __nv_bfloat162 x =
                      __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), fb);
                  w[i] = *reinterpret_cast<const uint32_t*>(&x);
                }
                tmem_st16(s_addr + e, w);
              }
              if (j < mine - 1) scale_output<D>(o_addr, f);
            }
            sum0 = add2(sum0, add0);
            sum1 = add2(sum1, add1);
            tmem_st16(s_addr + c / 2, pk);
          }
        } else {
          // Two passes: the maximum (masked scores go back in place), then the
          // weights.  (One pass, as above: 722 against 703 us for 8192 rows.)
          float mt = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 128; c += 64) {
            uint32_t r[64];
            tmem_ld64(s_addr + c, r);
            float* s = reinterpret_cast<float*>(r);
            if (edge) {
              hide_keys(s, rel - c);
              hide_keys(s + 32, rel - c - 32);
              tmem_st32(s_addr + c, r);
              tmem_st32(s_addr + c + 32, r + 32);
            }
            mt = fmaxf(mt, chunk_max<64>(s));
          }
          if (edge) tmem_wait_st();
          mt *= mul;
          if (j == mine - 1) {
            m = mt + kHeadroom;
          } else if (__any_sync(0xffffffffu, mt > m)) {
            const float f = raise_max(m, mt);
            l *= f;
            scale_output<D>(o_addr, f);
          }
#pragma unroll 1
          for (int c = 0; c < 128; c += 64) {
            uint32_t r[64], pk[32];
            tmem_ld64(s_addr + c, r);
            chunk_weights<64>(reinterpret_cast<const float*>(r), mul, m, pk, sum0, sum1);
            tmem_st32(s_addr + c / 2, pk);
          }
        }
        float a0, a1;
        unpack2(add2(sum0, sum1), a0, a1);
        l += a0 + a1;
        // Value rows behind the last key of the sequence, up to the product's end.
        if (n_k - k0 < kTileRows) {
          const int r0 = n_k - k0, r1 = min(kTileRows, (end - k0 + 15) & ~15);
          if (r0 < r1) {
            const uint32_t f = fill + 2 * (tiles - 1 - j) + 1;
            ok = pre_wait(bars, &bars.full[f % kStages], (f / kStages) & 1, a.status);
            if (!ok) break;
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
      fill += 2 * tiles;
      if (!ok) break;
      if (mine > 0) {
        ok = pre_wait(bars, &bars.o[t], used & 1, a.status);
        if (!ok) break;
        ++used;
        tc_fence_after();
      }
      // A row without a visible key has l = 0: its O, products of zeros, stays 0.
      const float inv = inv_or_zero(l);
      const uint64_t inv2 = pack2(inv, inv);
      // Four lanes exchange 16-byte parts of their rows, so that a store covers
      // 64 bytes of each of eight rows instead of 16 of 32.
      const int row4 = row & ~3, part = lane & 3;
      __nv_bfloat16* dst =
          static_cast<__nv_bfloat16*>(a.o) + (at - part * static_cast<int64_t>(a.q_heads)) * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32], w[4][4];
        if (mine > 0) {
          tmem_ld32(o_addr + c, o);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0u;
        }
        if (c == D - 32 && mine > 0) {
          tc_fence_before();
          mbar_arrive(&bars.o_empty[t]);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float x, y;
          unpack2(mul2(pack2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), inv2), x, y);
          const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
          w[i / 4][i % 4] = *reinterpret_cast<const uint32_t*>(&b);
        }
        // w[j] of lane i becomes part i of the row of lane j (of the four).
#pragma unroll
        for (int b = 1; b < 4; b <<= 1) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (j & b) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool up = part & b;
              const uint32_t got =
                  __shfl_xor_sync(0xffffffffu, up ? w[j][e] : w[j | b][e], b);
              if (up) w[j][e] = got; else w[j | b][e] = got;
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (sound && row4 + j < rows)
            *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(j) * a.q_heads * D + c + 8 * part) =
                make_uint4(w[j][0], w[j][1], w[j][2], w[j][3]);
      }
      if (live && a.lse != nullptr) a.lse[at] = row_lse(m, l);
    }
  }
  __syncwarp();  // the issuing lanes rejoin their warps
  tc_fence_before();
  __syncthreads();
  if (warp == kProducts) tmem_dealloc(tmem, 512);
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
  return encode_tile_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, 3, dims, strides, box);
}

// The grid: a block an item, at most 32 blocks an SM, which still lets claims
// even out what the items differ by.  (Uncapped, one prompt of 512 rows in a
// batch padded to 4096 sequences took 11 ms for the claims of empty ones, and
// 63 us capped.)
constexpr int kBlocksPerSm = 32;
template <int D, bool CAP, bool BIAS>
cudaError_t launch_tc(PrefillTcParams& p, cudaStream_t stream) {
  const cudaError_t e = ensure_max_smem<prefill_tc_kernel<D, CAP, BIAS>>();
  if (e != cudaSuccess) return e;
  const int block_rows = p.pair_heads ? kTileRows : 2 * kTileRows;
  const int64_t items = doc_blocks(p.a.rows_q, p.a.n_docs, block_rows, 1) *
                        (p.pair_heads ? p.a.q_heads / 2 : p.a.q_heads);
  const int64_t blocks = std::min<int64_t>(items, kBlocksPerSm * device_sm_count());
  p.capped = blocks < items;
  prefill_tc_kernel<D, CAP, BIAS>
      <<<static_cast<unsigned>(blocks), kPreThreads, PreShape<D>::kSmem, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_tc_opts(PrefillTcParams& p, cudaStream_t stream) {
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
  p.inject_polls = consume_wait_injection();
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
