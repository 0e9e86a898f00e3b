// Pieces of the dense attentions on the fifth-generation tensor cores (bf16;
// packed prompts, wf_prefill.cu, and drafted trees and windows over pages,
// wf_paged_umma.cuh): tensor-memory accesses, operand descriptors, the scores'
// mapping and mask, weights and the running maximum, all for 128-row tiles with
// one softmax thread a query row.
#pragma once

#include "wf_attn.cuh"
#include "wf_umma.cuh"

namespace wf {

namespace {

constexpr int kTileRows = 128;  // query rows of a tile, keys of a tile
constexpr float kRaise = 8.f;   // a maximum above the score that raised it (log2)

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

// The lowest n bits (none, or all 32, for n outside).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
}
// The keys of a chunk that a row sees, one bit a key: those below `end`; window:
// from `low` on, or below `sinks` (all relative to the chunk's first key).
template <bool WINDOW>
__device__ __forceinline__ uint32_t seen_keys(int end, int low, int sinks) {
  const uint32_t seen = low_bits(end);
  return WINDOW ? (seen & ~low_bits(low)) | low_bits(sinks) : seen;
}
// The keys of a chunk that are not seen are hidden: their scores become `with`.
// Bits of a register become predicates eight at once.
__device__ __forceinline__ void hide_keys(float* s, uint32_t seen, float with = -INFINITY) {
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

// Weights 2^(s mul - m), packed to bf16 (half a step, 2^-8 relative each: the type
// that the tensor cores take beside bf16 values; two parts of a weight would double the
// product with the values and the columns that it is read from); their sum, before that
// rounding, in fp32, in two parts.
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

// Rows whose new score exceeds the maximum raise it to kRaise above that
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
  m = mt + kRaise;
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

// Four lanes exchange 16-byte parts of their rows: w[j] of lane i becomes part i
// of the row of lane j (of the four), so that a store covers 64 bytes of each of
// eight rows instead of 16 of 32.
__device__ __forceinline__ void exchange_rows(uint32_t (&w)[4][4], int part) {
#pragma unroll
  for (int b = 1; b < 4; b <<= 1) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j & b) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool up = part & b;
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[j][e] : w[j | b][e], b);
        if (up) w[j][e] = got; else w[j | b][e] = got;
      }
    }
  }
}

}  // namespace

}  // namespace wf
