// Attention over packed sequences on the FMA pipes: fp32 inputs (bf16 ones
// run on the tensor cores, wf_prefill.cu).
//
// A row block is 64 rows of one key-value head: row r = i g + h is query i of
// the block's sequence at head h of the g query heads sharing the keys, so
// shared keys are read once for all of them.  256 threads as 16 x 16: thread
// (ty, tx) owns four rows and, of a 64-key tile, keys tx, tx + 16, ...; then
// of the output columns float4s tx, tx + 16.  One pass over the keys with the
// running maximum and sum; the weights pass through shared memory within a
// half warp.  32 heads, 2048 rows and keys, d = 128: 2490 us, 27.6 TFLOP/s of
// the pipes' 80.  At 119 KB of shared memory eight warps share an SM, whose
// chains of shared-memory reads and FMAs bound it: fetching the next tile into
// registers meanwhile (1 % less) or four weights a read (2 % more) changed
// little.
#include <algorithm>

#include "wf_attn.cuh"

namespace wf {

namespace {

constexpr int KT = 64;  // keys per tile

// The windowed kernel is launched early.
constexpr int read_of_window(bool window) { return window ? kReadOrdered : kReadConst; }

template <int D, int RT>
struct FmaSmem {
  float q[RT][D + 4];
  float k[KT][D + 4];
  float v[KT][D + 4];
  float p[RT][KT + 4];
};

// One row block's running state in registers.
template <int D, int RT>
struct FmaState {
  static constexpr int RPT = RT / 16;
  float m[RPT], l[RPT], o[RPT][D / 16];
  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) o[r][c] = 0.f;
    }
  }
};

// What a row block needs to know of its rows and sequence.
struct RowBlock {
  int row0, rows;  // first row and row count within the unit
  int g, n_q, len, prefix, head0;
  int window, sinks;  // window 0: none
  __device__ __forceinline__ int pos(int r) const { return len - n_q + (row0 + r) / g; }
  __device__ __forceinline__ int head(int r) const { return head0 + (row0 + r) % g; }
};

// One 64-key tile (keys key0 .. key0 + 63, staged in shared memory, rows past
// `len` zero) into the running state.
template <int D, int RT, bool WINDOW>
__device__ __forceinline__ void fma_tile(FmaSmem<D, RT>& s, const RowBlock& b,
                                         const ScoreOpts& o, int key0, FmaState<D, RT>& st) {
  constexpr int RPT = RT / 16;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float z[RPT][4];
#pragma unroll
  for (int r = 0; r < RPT; ++r)
#pragma unroll
    for (int j = 0; j < 4; ++j) z[r][j] = 0.f;
#pragma unroll 4
  for (int d = 0; d < D; d += 4) {
    float4 qv[RPT], kv[4];
#pragma unroll
    for (int r = 0; r < RPT; ++r) qv[r] = *reinterpret_cast<const float4*>(&s.q[ty * RPT + r][d]);
#pragma unroll
    for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(&s.k[tx + 16 * j][d]);
#pragma unroll
    for (int r = 0; r < RPT; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        z[r][j] = fmaf(qv[r].x, kv[j].x, z[r][j]);
        z[r][j] = fmaf(qv[r].y, kv[j].y, z[r][j]);
        z[r][j] = fmaf(qv[r].z, kv[j].z, z[r][j]);
        z[r][j] = fmaf(qv[r].w, kv[j].w, z[r][j]);
      }
  }
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    const int row = ty * RPT + r;
    const int pos = b.pos(row);
    const float slope = o.slopes != nullptr && row < b.rows
                            ? load_input<read_of_window(WINDOW)>(o.slopes + b.head(row))
                            : 0.f;
    float mx = st.m[r];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int key = key0 + tx + 16 * j;
      float x = z[r][j] * o.scale;
      if (o.cap > 0.f) x = o.cap * tanhf(x);
      x -= slope * kLog2e * fabsf(static_cast<float>(pos - key));
      bool seen = key < b.len && (!o.causal || key <= pos || key < b.prefix);
      if (WINDOW)
        seen = seen && (key < b.sinks ||
                        (pos - key < b.window && (o.causal || key - pos < b.window)));
      z[r][j] = seen ? x : -INFINITY;
      mx = fmaxf(mx, z[r][j]);
    }
#pragma unroll
    for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
    const float base = mx == -INFINITY ? 0.f : mx;
    const float corr = fast_exp2(st.m[r] - base);  // m = -inf: 0
    st.m[r] = mx;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float e = fast_exp2(z[r][j] - base);
      s.p[row][tx + 16 * j] = e;
      sum += e;
    }
#pragma unroll
    for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
    st.l[r] = st.l[r] * corr + sum;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) st.o[r][c] *= corr;
  }
  __syncwarp();
#pragma unroll 4
  for (int j = 0; j < KT; ++j) {
    float pv[RPT];
#pragma unroll
    for (int r = 0; r < RPT; ++r) pv[r] = s.p[ty * RPT + r][j];
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      const float4 vv = *reinterpret_cast<const float4*>(&s.v[j][tx * 4 + 64 * c]);
#pragma unroll
      for (int r = 0; r < RPT; ++r) {
        st.o[r][4 * c] = fmaf(pv[r], vv.x, st.o[r][4 * c]);
        st.o[r][4 * c + 1] = fmaf(pv[r], vv.y, st.o[r][4 * c + 1]);
        st.o[r][4 * c + 2] = fmaf(pv[r], vv.z, st.o[r][4 * c + 2]);
        st.o[r][4 * c + 3] = fmaf(pv[r], vv.w, st.o[r][4 * c + 3]);
      }
    }
  }
}

// Finished rows: O and lse of the unit's rows at o/lse rows (i * hq + head).
template <typename T, int D, int RT>
__device__ __forceinline__ void fma_store(const FmaState<D, RT>& st, const RowBlock& b, T* o,
                                          float* lse, int hq) {
  constexpr int RPT = RT / 16;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    const int row = ty * RPT + r;
    if (row >= b.rows) continue;
    const int64_t at = static_cast<int64_t>((b.row0 + row) / b.g) * hq + b.head(row);
    const float inv = inv_or_zero(st.l[r]);
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      float f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = st.o[r][4 * c + e] * inv;
      store4(o + at * D + tx * 4 + 64 * c, f);
    }
    if (lse != nullptr && tx == 0)
      lse[at] = row_lse(st.m[r], st.l[r]);
  }
}

template <int READ, typename T, int D, int RT>
__device__ __forceinline__ void fma_load_q(FmaSmem<D, RT>& s, const RowBlock& b, const T* q,
                                           int64_t stride) {
  static_assert(sizeof(T) == 4, "rows of fp32");
  constexpr int V = Elem<T>::kPer16B, C = D / V;
  for (int e = threadIdx.x; e < RT * C; e += kThreads) {
    const int r = e / C, c = e % C;
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < b.rows)
      f = load_input<READ>(reinterpret_cast<const float4*>(
          q + static_cast<int64_t>((b.row0 + r) / b.g) * stride + b.head(r) * D + c * V));
    *reinterpret_cast<float4*>(&s.q[r][c * V]) = f;
  }
}

// Stages one key or value row chunk (zero when src is null).
template <typename T, int D, int RT>
__device__ __forceinline__ void fma_stage(FmaSmem<D, RT>& s, int j, int c, const T* k, const T* v) {
  constexpr int V = Elem<T>::kPer16B;
  float f[V], h[V];
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = h[i] = 0.f;
  if (k != nullptr) {
    load16_f32(k + c * V, f);
    load16_f32(v + c * V, h);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    s.k[j][c * V + i] = f[i];
    s.v[j][c * V + i] = h[i];
  }
}

struct PrefillParams {
  PrefillArgs a;
  ScoreOpts o;
  int capped;  // 1: the grid has fewer blocks than row blocks there might be
};

template <typename T, int D, int RT, bool WINDOW>
__global__ void __launch_bounds__(kThreads) prefill_fma_kernel(PrefillParams p) {
  extern __shared__ float4 smem4[];
  FmaSmem<D, RT>& s = *reinterpret_cast<FmaSmem<D, RT>*>(smem4);
  const PrefillArgs& a = p.a;
  const int g = a.q_heads / a.kv_heads;
  const int kvh = blockIdx.y;
  constexpr int kRead = read_of_window(WINDOW);
  if (WINDOW) wait_for_primary();
  if (blockIdx.x == 0 && kvh == 0) {
    check_offsets<kRead>(a.cu_q, a.n_docs, a.rows_q, a.status, threadIdx.x, kThreads);
    check_offsets<kRead>(a.cu_k, a.n_docs, a.rows_k, a.status, threadIdx.x, kThreads);
  }
  DocCursor cursor = {0, 0};
  const int64_t total = p.capped ? doc_total<kRead>(a, RT, g) : gridDim.x;
  for (int64_t at = blockIdx.x; at < total; at += gridDim.x) {
    DocBlock d;
    if (!find_doc_block<kRead>(a, at, RT, g, cursor, &d)) return;
    if (at != blockIdx.x) __syncthreads();  // the last block's rows have been read
    RowBlock b;
    b.g = g;
    b.n_q = d.n_q;
    b.len = d.n_k;
    b.prefix = p.o.prefix != nullptr ? load_input<kRead>(p.o.prefix + d.doc) : 0;
    b.row0 = d.block * RT;
    b.rows = min(RT, d.n_q * g - b.row0);
    b.head0 = kvh * g;
    fma_load_q<kRead, T, D, RT>(s, b, static_cast<const T*>(a.q) + d.q0 * a.q_stride, a.q_stride);
    FmaState<D, RT> st;
    st.reset();
    int end = visible_end(b.len, b.pos(b.rows - 1), p.o.causal, b.prefix);
    // Window: the tiles between the first tokens and the first row's window are
    // passed over, and those behind the last one's.
    int sinks_end = 0, low = 0;
    b.window = a.window;
    b.sinks = a.sinks;
    if (WINDOW) {
      const int last = b.pos(b.rows - 1);
      sinks_end = min(a.sinks, b.len);
      low = max(0, b.pos(0) - a.window + 1) / KT * KT;
      if (!p.o.causal && a.window < b.len - last) end = max(last + a.window, sinks_end);
    }
    const T* kb = static_cast<const T*>(a.k) + d.k0 * a.k_stride + kvh * D;
    const T* vb = static_cast<const T*>(a.v) + d.k0 * a.v_stride + kvh * D;
    if constexpr (WINDOW) {
      // A window's few tiles are bound by the latency of their copies: the next tile
      // comes into registers while this one is worked on (one prompt of 4001 rows,
      // window 256, 2 heads, d = 64: 75 -> 70 us, the reads of shared memory bound it).
      constexpr int V = Elem<T>::kPer16B, C = D / V, kMine = KT * C / kThreads;
      uint4 kr[kMine], vr[kMine];
      const auto fetch = [&](int key0) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          const int e = threadIdx.x + i * kThreads, j = e / C, c = e % C, key = key0 + j;
          kr[i] = vr[i] = make_uint4(0u, 0u, 0u, 0u);
          if (key >= b.len) continue;
          kr[i] = load_input<kRead>(reinterpret_cast<const uint4*>(kb + key * a.k_stride) + c);
          vr[i] = load_input<kRead>(reinterpret_cast<const uint4*>(vb + key * a.v_stride) + c);
        }
      };
      const auto next = [&](int key0) {  // the next tile that some row sees
        key0 += KT;
        return key0 >= sinks_end && key0 < low ? low : key0;
      };
      int key0 = sinks_end > 0 ? 0 : low;
      if (key0 < end) fetch(key0);
      for (; key0 < end; key0 = next(key0)) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          const int e = threadIdx.x + i * kThreads, j = e / C, c = e % C;
          *reinterpret_cast<uint4*>(&s.k[j][c * V]) = kr[i];
          *reinterpret_cast<uint4*>(&s.v[j][c * V]) = vr[i];
        }
        __syncthreads();
        if (next(key0) < end) fetch(next(key0));
        fma_tile<D, RT, WINDOW>(s, b, p.o, key0, st);
      }
      end = 0;
    }
    for (int key0 = 0; key0 < end; key0 += KT) {
      __syncthreads();
      constexpr int C = D / Elem<T>::kPer16B;
      for (int e = threadIdx.x; e < KT * C; e += kThreads) {
        const int j = e / C, c = e % C, key = key0 + j;
        const bool in = key < b.len;
        fma_stage<T, D, RT>(s, j, c, in ? kb + key * a.k_stride : nullptr,
                            in ? vb + key * a.v_stride : nullptr);
      }
      __syncthreads();
      fma_tile<D, RT, WINDOW>(s, b, p.o, key0, st);
    }
    const int64_t base = d.q0 * a.q_heads;
    fma_store<T, D, RT>(st, b, static_cast<T*>(a.o) + base * D,
                        a.lse != nullptr ? a.lse + base : nullptr, a.q_heads);
  }
}

template <typename T, int D, bool WINDOW>
cudaError_t launch_prefill_typed(PrefillParams& p, cudaStream_t stream) {
  constexpr int RT = 64;
  const cudaError_t e = ensure_max_smem<prefill_fma_kernel<T, D, RT, WINDOW>>();
  if (e != cudaSuccess) return e;
  const int64_t blocks = doc_blocks(p.a.rows_q, p.a.n_docs, RT, p.a.q_heads / p.a.kv_heads);
  // At most about 32 CTAs an SM (one runs at a time), each with every so many
  // row blocks.
  const int64_t most = std::max(1, 32 * device_sm_count() / p.a.kv_heads);
  p.capped = most < blocks;
  const dim3 grid(static_cast<unsigned>(std::min(blocks, most)), p.a.kv_heads);
  if constexpr (WINDOW)
    return launch_early(prefill_fma_kernel<T, D, RT, WINDOW>, grid, kThreads,
                        sizeof(FmaSmem<D, RT>), stream, p);
  prefill_fma_kernel<T, D, RT, WINDOW><<<grid, kThreads, sizeof(FmaSmem<D, RT>), stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefill_fma(const PrefillArgs& a, cudaStream_t stream) {
  PrefillParams p;
  p.a = a;
  p.o = score_opts(a.scale, a.softcap, a.causal, a.prefix, a.slopes);
  if (a.window > 0)
    return a.head_dim == 128 ? launch_prefill_typed<float, 128, true>(p, stream)
                             : launch_prefill_typed<float, 64, true>(p, stream);
  return a.head_dim == 128 ? launch_prefill_typed<float, 128, false>(p, stream)
                           : launch_prefill_typed<float, 64, false>(p, stream);
}

}  // namespace wf
