// New rows into a paged cache, with the position rotation on the way.
//
// Each new row t of sequence s (cu_rows[s] <= t < cu_rows[s + 1]) takes cache
// position n = cache_len[s] + (t - cu_rows[s]): row n % page_size of page
// table[s][n / page_size].  Pages are [n_pages, kv_heads, page_size, d], so
// one head's rows of a page are contiguous.  Keys (and queries) are rotated,
// pair i of the first rotary_dim channels by the angle p f_i.
//
// Angles.  The caller's f_i become turns per position, f_i / 2π, as 64-bit
// binary fractions F_i, rounded to their last place.  p F_i mod 2^64 is then
// the angle's fraction of a turn, reduced without error, off by about p 2^-65
// turns for F_i's sake, and its top 54 bits go to the sine and cosine: no angle
// is ever formed whose rounding grows with p.
//
// HBM-bound: every byte is read once and written once.  One thread moves two
// 16-byte chunks that rotate together ((c, c + r/2) of the halves form,
// neighbours otherwise); a block takes 32 * ITERS consecutive (row, head)
// lines of the flattened [rows][q heads, k heads, v heads] order, issues all
// its loads first, resolves its rows' pages (one warp a row) and forms their
// sines once for all heads while the loads fly.  Four lines a thread keep
// 128 bytes in flight; below 4 blocks per SM, one line a thread, so that a
// decoding step's few rows spread over more SMs.
#include <algorithm>

#include "wf_common.cuh"
#include "wf_internal.h"

namespace wf {

namespace {

struct AppendParams {
  AppendArgs a;
  RopeTurns turns;
  int page_shift;  // log2 page_size
};

// The sequence of row t: the last s < n_seqs with cu[s] <= t, or -1 when t
// is at or behind cu[n_seqs] (or before cu[0]).  Whole warp, 32-way search.
__device__ __forceinline__ int row_sequence(const int32_t* cu, int n_seqs, int t) {
  const int lane = threadIdx.x & 31;
  if (t < __ldg(cu) || t >= __ldg(cu + n_seqs)) return -1;
  int lo = 0, n = n_seqs;  // cu[lo] <= t, the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lo + lane * step;
    const bool below = lane * step < n && __ldg(cu + at) <= t;
    const int k = 31 - __clz(__ballot_sync(0xffffffffu, below) | 1u);
    const int left = n - k * step;
    lo += k * step;
    n = min(step, left);
  }
  return lo;
}

template <typename T>
__device__ __forceinline__ uint4 pack16(const float* f);
template <>
__device__ __forceinline__ uint4 pack16<__nv_bfloat16>(const float* f) {
  uint4 v;
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return v;
}
template <>
__device__ __forceinline__ uint4 pack16<float>(const float* f) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                    __float_as_uint(f[3]));
}

struct TokenInfo {
  int64_t line;  // first cache line index ((page * kv_heads) * page_size + row), -1: no write
  int32_t pos;   // rotation position
  int32_t live;  // row belongs to a sequence
};

template <typename T, int D, int ITERS>
__global__ void __launch_bounds__(kThreads, ITERS == 1 ? 6 : 4)
    append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int V = Elem<T>::kPer16B;     // elements per chunk
  constexpr int C2 = D / (2 * V);         // chunk pairs per line
  constexpr int LANES = kThreads / C2;    // lines per pass
  constexpr int LINES = LANES * ITERS;    // lines per block
  // Cosines and sines of the block's rows, two pairs a float4: those of chunk
  // pair c lie C2 apart, so that the threads of a line read side by side.
  extern __shared__ float4 s_cs[];        // [tokens][V / 2][C2]
  __shared__ TokenInfo s_tok[LINES + 1];
  const AppendArgs& a = p.a;
  const int qh = a.q != nullptr ? a.q_heads : 0;
  const int per_row = qh + 2 * a.kv_heads;
  const int64_t total = static_cast<int64_t>(a.rows) * per_row;
  const int64_t line0 = static_cast<int64_t>(blockIdx.x) * LINES;
  // Row and line within it of the block's first line; every other line of the
  // block is a 32-bit step away.
  const int t0 = line0 >> 32 == 0
                     ? static_cast<int>(static_cast<uint32_t>(line0) / static_cast<uint32_t>(per_row))
                     : static_cast<int>(line0 / per_row);
  const uint32_t rest = static_cast<uint32_t>(line0 - static_cast<int64_t>(t0) * per_row);
  const int lines = static_cast<int>(min(static_cast<int64_t>(LINES), total - line0));
  const int n_tok = static_cast<int>((rest + lines - 1) / static_cast<uint32_t>(per_row)) + 1;
  const int c = threadIdx.x % C2;
  const int rot_pairs = a.rotary_dim / (2 * V);  // rotated chunk pairs per line
  // The two chunks of this thread: halves (c, c + r/2V), else neighbours.
  const bool rotate = c < rot_pairs;
  const bool halves = rotate && !a.interleaved;
  const int ca = halves ? c : 2 * c;
  const int cb = halves ? c + rot_pairs : 2 * c + 1;

  uint4 xa[ITERS], xb[ITERS];
  int tok[ITERS], head[ITERS];  // row within the block, line within the row (-1: none)
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    const int line = i * LANES + threadIdx.x / C2;
    const uint32_t at = rest + line;
    tok[i] = static_cast<int>(at / static_cast<uint32_t>(per_row));
    head[i] = line < lines ? static_cast<int>(at) - tok[i] * per_row : -1;
    if (line < lines) {
      const int64_t t = t0 + tok[i];
      const int h = head[i];
      const T* src = h < qh ? static_cast<const T*>(a.q) + t * a.q_stride + h * D
                     : h < qh + a.kv_heads
                         ? static_cast<const T*>(a.k) + t * a.k_stride + (h - qh) * D
                         : static_cast<const T*>(a.v) + t * a.v_stride + (h - qh - a.kv_heads) * D;
      // Ordinary loads: the queries may be rotated in place.
      xa[i] = ld16_stream(src + ca * V);
      xb[i] = ld16_stream(src + cb * V);
    }
  }

  for (int i = threadIdx.x >> 5; i < n_tok; i += kWarps) {
    const int t = t0 + i;
    const int s = row_sequence(a.cu_rows, a.n_seqs, t);
    if ((threadIdx.x & 31) == 0) {
      TokenInfo info = {-1, 0, 0};
      if (s >= 0) {
        info.live = 1;
        const int64_t n = static_cast<int64_t>(__ldg(a.cache_len + s)) + (t - __ldg(a.cu_rows + s));
        info.pos = a.positions != nullptr ? __ldg(a.positions + t) : static_cast<int32_t>(n);
        const int64_t slot = n >> p.page_shift;
        int page = -1;
        if (n >= 0 && slot < a.table_pages)
          page = __ldg(a.table + static_cast<int64_t>(s) * a.table_pages + slot);
        if (page >= 0 && page < a.n_pages)
          info.line = static_cast<int64_t>(page) * a.kv_heads * a.page_size +
                      (n & (a.page_size - 1));
        else
          raise_flag(a.status, WF_DEV_BAD_INDEX);
      }
      s_tok[i] = info;
    }
  }
  __syncthreads();
  const int half = a.rotary_dim / 2;
  for (int e = threadIdx.x; e < n_tok * half; e += kThreads) {
    const int i = e / half, j = e - i * half;
    // The fraction of a turn, in [-1/2, 1/2): its first 24 bits as half turns
    // (exact in fp32), the rest (below 2^-25 half turns) by the first term of
    // the sine's and cosine's series.  At the end of the range the first part
    // comes out as -1/2 turn, with the rest below 0.
    const uint64_t frac = static_cast<uint64_t>(static_cast<int64_t>(s_tok[i].pos)) * p.turns.f[j];
    const int32_t head = static_cast<int32_t>(static_cast<int64_t>(frac + (1ull << 38)) >> 39);
    const int64_t rest = static_cast<int64_t>(frac - (static_cast<uint64_t>(head) << 39));
    float sn, cs;
    sincospif(static_cast<float>(head) * 0x1p-24f, &sn, &cs);
    const float d = static_cast<float>(static_cast<int32_t>(rest >> 8)) * (0x1p-55f * 3.14159265f);
    const float sn0 = sn;
    sn = fmaf(d, cs, sn);
    cs = fmaf(-d, sn0, cs);
    reinterpret_cast<float2*>(s_cs + (i * (V / 2) + (j % V) / 2) * C2 + j / V)[j % 2] =
        make_float2(cs, sn);
  }
  __syncthreads();

#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    if (head[i] < 0) continue;
    const int64_t t = t0 + tok[i];
    int h = head[i];
    const TokenInfo info = s_tok[tok[i]];
    if (!info.live) continue;
    uint4 ya = xa[i], yb = xb[i];
    if (rotate && h < qh + a.kv_heads) {
      float fa[V], fb[V];
      widen16(ya, static_cast<const T*>(nullptr), fa);
      widen16(yb, static_cast<const T*>(nullptr), fb);
      const float4* cs = s_cs + tok[i] * (V / 2) * C2 + c;
      if (halves) {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          const float4 w = cs[e / 2 * C2];
          const float x0 = fa[e], y0 = fb[e], x1 = fa[e + 1], y1 = fb[e + 1];
          fa[e] = x0 * w.x - y0 * w.y;
          fb[e] = x0 * w.y + y0 * w.x;
          fa[e + 1] = x1 * w.z - y1 * w.w;
          fb[e + 1] = x1 * w.w + y1 * w.z;
        }
      } else {
        // Pairs 0 .. V/2 - 1 of the thread lie in chunk a, the rest in b.
        const auto turn = [](float& x, float& y, float cs, float sn) {
          const float u = x;
          x = u * cs - y * sn;
          y = u * sn + y * cs;
        };
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          const float4 w = cs[e / 2 * C2];
          float* f = e < V / 2 ? fa : fb;
          const int o = 2 * (e % (V / 2));
          turn(f[o], f[o + 1], w.x, w.y);
          turn(f[o + 2], f[o + 3], w.z, w.w);
        }
      }
      ya = pack16<T>(fa);
      yb = pack16<T>(fb);
    }
    T* dst = nullptr;
    if (h < qh) {
      dst = static_cast<T*>(a.q_out) + (t * qh + h) * D;
    } else {
      h -= qh;
      const bool is_k = h < a.kv_heads;
      if (!is_k) h -= a.kv_heads;
      if (is_k && a.k_out != nullptr) {
        T* ko = static_cast<T*>(a.k_out) + (t * a.kv_heads + h) * D;
        *reinterpret_cast<uint4*>(ko + ca * V) = ya;
        *reinterpret_cast<uint4*>(ko + cb * V) = yb;
      }
      if (info.line < 0) continue;
      dst = static_cast<T*>(is_k ? a.k_pages : a.v_pages) +
            (info.line + static_cast<int64_t>(h) * a.page_size) * D;
    }
    *reinterpret_cast<uint4*>(dst + ca * V) = ya;
    *reinterpret_cast<uint4*>(dst + cb * V) = yb;
  }
}

template <typename T, int D, int ITERS>
cudaError_t launch_iters(const AppendParams& p, cudaStream_t stream) {
  constexpr int LINES = kThreads / (D / (2 * Elem<T>::kPer16B)) * ITERS;
  const int per_row = (p.a.q != nullptr ? p.a.q_heads : 0) + 2 * p.a.kv_heads;
  const int64_t total = static_cast<int64_t>(p.a.rows) * per_row;
  const size_t tokens = (LINES - 1 + per_row - 1) / per_row + 1;
  const size_t smem = p.a.rotary_dim > 0 ? tokens * (D / 2) * sizeof(float2) : 0;
  const cudaError_t e = ensure_max_smem<append_kernel<T, D, ITERS>>();
  if (e != cudaSuccess) return e;
  append_kernel<T, D, ITERS>
      <<<static_cast<unsigned>((total + LINES - 1) / LINES), kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_typed(const AppendParams& p, cudaStream_t stream) {
  constexpr int LANES = kThreads / (D / (2 * Elem<T>::kPer16B));
  const int per_row = (p.a.q != nullptr ? p.a.q_heads : 0) + 2 * p.a.kv_heads;
  const int64_t total = static_cast<int64_t>(p.a.rows) * per_row;
  if (total >= static_cast<int64_t>(LANES) * 4 * 4 * device_sm_count())
    return launch_iters<T, D, 4>(p, stream);
  return launch_iters<T, D, 1>(p, stream);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, const RopeTurns& turns, cudaStream_t stream) {
  AppendParams p;
  p.a = a;
  p.turns = turns;
  p.page_shift = 0;
  while ((1 << p.page_shift) < a.page_size) ++p.page_shift;
  if (a.dtype == WF_BF16) {
    if (a.head_dim == 128) return launch_typed<__nv_bfloat16, 128>(p, stream);
    return launch_typed<__nv_bfloat16, 64>(p, stream);
  }
  if (a.head_dim == 128) return launch_typed<float, 128>(p, stream);
  return launch_typed<float, 64>(p, stream);
}

}  // namespace wf
