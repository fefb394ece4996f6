// Attention over packed sequences on the CUDA cores, forward and backward:
// fp32 storage, and bf16 tensors whose head size, alignment or strides the
// tensor-core kernels do not take.  Every product and sum is fp32.
//
//   s = scale q k^T (masked), lse = log sum e^s, p = e^(s - lse), o = p v
//   delta = sum_d do o,  dv = p^T do,  ds = p (do v^T - delta),
//   dq = scale ds k,  dk = scale ds^T q
//
// A CTA of 256 threads owns a tile of BT rows of one head (queries in the
// forward and in dq, keys in dk/dv) and walks the tiles of the other side,
// so every sum has one owner and a fixed order: no atomics, and dk, dv of a
// shared key head are summed over its query heads inside the CTA.  The
// backward is one launch: the first blocks own key tiles, the others query
// tiles, and each forms the delta of the rows it needs while it loads them.
// Thread (ty, tx) of 16 x 16 holds BT/16 rows x BT/16 columns of the score
// tile and, of the outputs, BT/16 rows x groups of 4 columns 64 apart.  Every
// operand is read from shared memory as float4 (rows padded by 4 words so that
// 8 lanes' reads fall into different banks): 12 (20) wavefronts of LDS for 64
// (128) warp instructions of FFMA in the two products of a 64 x 64 tile.
// Measured, one causal fp32 sequence of 4,096 tokens, 32/8 heads of 128: 5.6 ms
// (25 TFLOP/s over the unmasked scores) forward, 17.2 ms (20, and 28 with the
// scores and do v^T that dq and dk/dv each make) backward, of some 80 that the
// multiply-add units give.  Nothing is saturated: the multiply-add pipe is busy
// 35% (backward 41) of the cycles, shared memory 48 (53), the issue slots 49 (55).
// The bound is latency: the tiles' shared memory (119 and 170 KB) leaves one CTA
// per SM, two warps to a scheduler, and they wait for the scalar loads of a tile,
// which nothing overlaps, for shared memory and for each other's barriers.
#include <cmath>

#include "attn_common.cuh"

namespace ftk {

namespace {

constexpr int kThreads = 256;

// Loads rows [row0, row0 + BT) of one head into s (row stride ld words, D
// padded with zeros to DP; rows at or past len zeroed).
template <typename T, int BT>
__device__ __forceinline__ void load_rows(float *s, int ld, const T *base, int64_t stride, int row0,
                                          int len, int D, int DP) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int r = ty; r < BT; r += 16) {
    const bool in = row0 + r < len;
    const T *p = base + (int64_t)(row0 + r) * stride;
    for (int d = tx; d < DP; d += 16) s[r * ld + d] = (in && d < D) ? to_float(p[d]) : 0.f;
  }
}

// acc[i][j] = sum_d a[ty TM + i][d] b[tx + 16 j][d]
template <int TM>
__device__ __forceinline__ void rows_dot(float (&acc)[TM][TM], const float *a, const float *b,
                                         int ld, int DP) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = 0.f;
  for (int d = 0; d < DP; d += 4) {
    float4 x[TM], y[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i)
      x[i] = *reinterpret_cast<const float4 *>(a + (ty * TM + i) * ld + d);
#pragma unroll
    for (int j = 0; j < TM; ++j)
      y[j] = *reinterpret_cast<const float4 *>(b + (tx + 16 * j) * ld + d);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        float s = acc[i][j];
        s = fmaf(x[i].x, y[j].x, s);
        s = fmaf(x[i].y, y[j].y, s);
        s = fmaf(x[i].z, y[j].z, s);
        acc[i][j] = fmaf(x[i].w, y[j].w, s);
      }
  }
}

// out[i][n][e] += sum_c p[ty TM + i][c] b[c][4 tx + 64 n + e], c < nc (p and b
// hold zeros, or products that are zero, up to the next multiple of 4)
template <int TM, int NN>
__device__ __forceinline__ void rows_mul(float (&out)[TM][NN][4], const float *p, int ldp,
                                         const float *b, int ld, int nc, int DP) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  if (4 * tx >= DP) return;
  for (int c = 0; c < nc; c += 4) {
    float x[TM][4];
#pragma unroll
    for (int i = 0; i < TM; ++i)
      *reinterpret_cast<float4 *>(x[i]) =
          *reinterpret_cast<const float4 *>(p + (ty * TM + i) * ldp + c);
#pragma unroll
    for (int n = 0; n < NN; ++n) {
      const int d = 4 * tx + 64 * n;
      if (d >= DP) break;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float4 y = *reinterpret_cast<const float4 *>(b + (c + u) * ld + d);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          out[i][n][0] = fmaf(x[i][u], y.x, out[i][n][0]);
          out[i][n][1] = fmaf(x[i][u], y.y, out[i][n][1]);
          out[i][n][2] = fmaf(x[i][u], y.z, out[i][n][2]);
          out[i][n][3] = fmaf(x[i][u], y.w, out[i][n][3]);
        }
      }
    }
  }
}

template <typename T, int TM, int NN>
__device__ __forceinline__ void store_rows(T *base, int64_t stride, int row0, int len, int D,
                                           const float (&out)[TM][NN][4], const float (&f)[TM]) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int r = row0 + ty * TM + i;
    if (r >= len) continue;
    T *p = base + (int64_t)r * stride;
#pragma unroll
    for (int n = 0; n < NN; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = 4 * tx + 64 * n + e;
        if (d < D) p[d] = from_float<T>(out[i][n][e] * f[i]);
      }
  }
}

template <int TM, int NN> __device__ __forceinline__ void clear(float (&out)[TM][NN][4]) {
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int n = 0; n < NN; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) out[i][n][e] = 0.f;
}

// The sum (or maximum) over the 16 lanes that hold one row.
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// load_rows of do that also leaves delta[r] = sum_d do o of its rows in s_delta.
template <typename T, int BT>
__device__ __forceinline__ void load_rows_delta(float *s, float *s_delta, int ld, const T *base,
                                                int64_t stride, const T *o, int64_t ld_o, int row0,
                                                int len, int D, int DP) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int r = ty; r < BT; r += 16) {
    const bool in = row0 + r < len;
    const T *p = base + (int64_t)(row0 + r) * stride, *po = o + (int64_t)(row0 + r) * ld_o;
    float dot = 0.f;
    for (int d = tx; d < DP; d += 16) {
      const bool real = in && d < D;
      const float g = real ? to_float(p[d]) : 0.f;
      if (real) dot = fmaf(g, to_float(po[d]), dot);
      s[r * ld + d] = g;
    }
    dot = row_sum(dot);
    if (tx == 0) s_delta[r] = dot;
  }
}

template <typename T, int BT, int DMAX>
__global__ void __launch_bounds__(kThreads)
attn_fwd_generic(const AttnArgs a, int slots) {
  constexpr int TM = BT / 16, NN = DMAX / 64, LDP = BT + 4;
  extern __shared__ float sm[];
  pdl_wait();
  pdl_trigger();
  if (attn_skipped(a.skip)) return;
  const int DP = (a.D + 3) & ~3, ld = DP + 4;
  float *Qs = sm, *Ks = Qs + BT * ld, *Vs = Ks + BT * ld, *Ps = Vs + BT * ld;
  // heads run fastest; tiles from the last one back, whose rows see most keys
  const int h = blockIdx.x % a.Hq, slot = slots - 1 - (int)(blockIdx.x / a.Hq);
  const SeqTile t = seq_tile(slot, a.cu, a.B, (int)a.T, BT);
  if (t.len == 0) return;
  const int hk = h / (a.Hq / a.Hkv);
  const T *q = (const T *)a.q + t.start * a.ld_q + (int64_t)h * a.D;
  const T *k = (const T *)a.k + t.start * a.ld_k + (int64_t)hk * a.D;
  const T *v = (const T *)a.v + t.start * a.ld_v + (int64_t)hk * a.D;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  load_rows<T, BT>(Qs, ld, q, a.ld_q, t.row0, t.len, a.D, DP);
  float out[TM][NN][4], m[TM], l[TM];
  clear(out);
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
  }
  const int end = a.causal ? min(t.len, t.row0 + BT) : t.len;
  for (int c0 = 0; c0 < end; c0 += BT) {
    __syncthreads();
    load_rows<T, BT>(Ks, ld, k, a.ld_k, c0, t.len, a.D, DP);
    load_rows<T, BT>(Vs, ld, v, a.ld_v, c0, t.len, a.D, DP);
    __syncthreads();
    float s[TM][TM];
    rows_dot<TM>(s, Qs, Ks, ld, DP);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int r = t.row0 + ty * TM + i;
      float mx = m[i];
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const int c = c0 + tx + 16 * j;
        const bool see = c < t.len && (!a.causal || c <= r);
        s[i][j] = see ? s[i][j] * a.scale : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
      mx = row_max(mx);
      // -inf while every key so far scored -inf (infinite keys, an overflow)
      const float off = mx == -INFINITY ? 0.f : mx;
      const float f = expf(m[i] - off);
      m[i] = mx;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const float p = expf(s[i][j] - off);
        sum += p;
        Ps[(ty * TM + i) * LDP + tx + 16 * j] = p;
      }
      l[i] = l[i] * f + row_sum(sum);
#pragma unroll
      for (int n = 0; n < NN; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) out[i][n][e] *= f;
    }
    __syncthreads();
    rows_mul<TM, NN>(out, Ps, LDP, Vs, ld, min(BT, t.len - c0), DP);
  }
  float inv[TM];
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    inv[i] = 1.f / l[i];
    const int r = t.row0 + ty * TM + i;
    if (a.lse && tx == 0 && r < t.len) a.lse[(int64_t)h * a.T + t.start + r] = m[i] + logf(l[i]);
  }
  T *o = (T *)a.o + t.start * a.ld_o + (int64_t)h * a.D;
  store_rows<T, TM, NN>(o, a.ld_o, t.row0, t.len, a.D, out, inv);
}

// dq of one query tile.
template <typename T, int BT, int DMAX>
__device__ __forceinline__ void dq_tile(const AttnArgs &a, float *sm, int h, int slot) {
  constexpr int TM = BT / 16, NN = DMAX / 64, LDP = BT + 4;
  const int DP = (a.D + 3) & ~3, ld = DP + 4;
  float *Qs = sm, *Gs = Qs + BT * ld, *Ks = Gs + BT * ld, *Vs = Ks + BT * ld, *Ds = Vs + BT * ld;
  float *Dl = Ds + BT * LDP;
  const SeqTile t = seq_tile(slot, a.cu, a.B, (int)a.T, BT);
  if (t.len == 0) return;
  const int hk = h / (a.Hq / a.Hkv);
  const T *q = (const T *)a.q + t.start * a.ld_q + (int64_t)h * a.D;
  const T *g = (const T *)a.do_ + t.start * a.ld_do + (int64_t)h * a.D;
  const T *o = (const T *)a.o + t.start * a.ld_o + (int64_t)h * a.D;
  const T *k = (const T *)a.k + t.start * a.ld_k + (int64_t)hk * a.D;
  const T *v = (const T *)a.v + t.start * a.ld_v + (int64_t)hk * a.D;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  load_rows<T, BT>(Qs, ld, q, a.ld_q, t.row0, t.len, a.D, DP);
  load_rows_delta<T, BT>(Gs, Dl, ld, g, a.ld_do, o, a.ld_o, t.row0, t.len, a.D, DP);
  float out[TM][NN][4], lse[TM], f[TM];
  clear(out);
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int r = t.row0 + ty * TM + i;
    lse[i] = r < t.len ? a.lse[(int64_t)h * a.T + t.start + r] : 0.f;
    f[i] = a.scale;
  }
  const int end = a.causal ? min(t.len, t.row0 + BT) : t.len;
  for (int c0 = 0; c0 < end; c0 += BT) {
    __syncthreads();
    load_rows<T, BT>(Ks, ld, k, a.ld_k, c0, t.len, a.D, DP);
    load_rows<T, BT>(Vs, ld, v, a.ld_v, c0, t.len, a.D, DP);
    __syncthreads();
    float s[TM][TM], dp[TM][TM];
    rows_dot<TM>(s, Qs, Ks, ld, DP);
    rows_dot<TM>(dp, Gs, Vs, ld, DP);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int r = t.row0 + ty * TM + i;
      const float delta = Dl[ty * TM + i];
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const int c = c0 + tx + 16 * j;
        const bool see = c < t.len && r < t.len && (!a.causal || c <= r);
        const float p = see ? expf(fmaf(s[i][j], a.scale, -lse[i])) : 0.f;
        Ds[(ty * TM + i) * LDP + tx + 16 * j] = see ? p * (dp[i][j] - delta) : 0.f;
      }
    }
    __syncthreads();
    rows_mul<TM, NN>(out, Ds, LDP, Ks, ld, min(BT, t.len - c0), DP);
  }
  T *dq = (T *)a.dq + t.start * a.ld_dq + (int64_t)h * a.D;
  store_rows<T, TM, NN>(dq, a.ld_dq, t.row0, t.len, a.D, out, f);
}

// dk and dv of one key tile.  Rows are keys, columns queries: the score tile is
// transposed.
template <typename T, int BT, int DMAX>
__device__ __forceinline__ void dkv_tile(const AttnArgs &a, float *sm, int hk, int slot) {
  constexpr int TM = BT / 16, NN = DMAX / 64, LDP = BT + 4;
  const int DP = (a.D + 3) & ~3, ld = DP + 4;
  float *Ks = sm, *Vs = Ks + BT * ld, *Qs = Vs + BT * ld, *Gs = Qs + BT * ld, *Ps = Gs + BT * ld;
  float *Ds = Ps + BT * LDP, *Ls = Ds + BT * LDP, *Dl = Ls + BT;
  const SeqTile t = seq_tile(slot, a.cu, a.B, (int)a.T, BT);
  if (t.len == 0) return;
  const int G = a.Hq / a.Hkv;
  const T *k = (const T *)a.k + t.start * a.ld_k + (int64_t)hk * a.D;
  const T *v = (const T *)a.v + t.start * a.ld_v + (int64_t)hk * a.D;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  load_rows<T, BT>(Ks, ld, k, a.ld_k, t.row0, t.len, a.D, DP);
  load_rows<T, BT>(Vs, ld, v, a.ld_v, t.row0, t.len, a.D, DP);
  float dk[TM][NN][4], dv[TM][NN][4], fk[TM], fv[TM];
  clear(dk);
  clear(dv);
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    fk[i] = a.scale;
    fv[i] = 1.f;
  }
  for (int h = hk * G; h < (hk + 1) * G; ++h) {
    const T *q = (const T *)a.q + t.start * a.ld_q + (int64_t)h * a.D;
    const T *g = (const T *)a.do_ + t.start * a.ld_do + (int64_t)h * a.D;
    const T *o = (const T *)a.o + t.start * a.ld_o + (int64_t)h * a.D;
    for (int c0 = a.causal ? t.row0 : 0; c0 < t.len; c0 += BT) {
      __syncthreads();
      load_rows<T, BT>(Qs, ld, q, a.ld_q, c0, t.len, a.D, DP);
      load_rows_delta<T, BT>(Gs, Dl, ld, g, a.ld_do, o, a.ld_o, c0, t.len, a.D, DP);
      if (threadIdx.x < BT) {
        const int c = c0 + threadIdx.x;
        Ls[threadIdx.x] = c < t.len ? a.lse[(int64_t)h * a.T + t.start + c] : 0.f;
      }
      __syncthreads();
      float s[TM][TM], dp[TM][TM];
      rows_dot<TM>(s, Ks, Qs, ld, DP);
      rows_dot<TM>(dp, Vs, Gs, ld, DP);
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const int r = t.row0 + ty * TM + i;
#pragma unroll
        for (int j = 0; j < TM; ++j) {
          const int cc = tx + 16 * j, c = c0 + cc;
          const bool see = c < t.len && r < t.len && (!a.causal || r <= c);
          const float p = see ? expf(fmaf(s[i][j], a.scale, -Ls[cc])) : 0.f;
          Ps[(ty * TM + i) * LDP + cc] = p;
          Ds[(ty * TM + i) * LDP + cc] = see ? p * (dp[i][j] - Dl[cc]) : 0.f;
        }
      }
      __syncthreads();
      const int nc = min(BT, t.len - c0);
      rows_mul<TM, NN>(dv, Ps, LDP, Gs, ld, nc, DP);
      rows_mul<TM, NN>(dk, Ds, LDP, Qs, ld, nc, DP);
    }
  }
  T *pk = (T *)a.dk + t.start * a.ld_dk + (int64_t)hk * a.D;
  T *pv = (T *)a.dv + t.start * a.ld_dv + (int64_t)hk * a.D;
  store_rows<T, TM, NN>(pk, a.ld_dk, t.row0, t.len, a.D, dk, fk);
  store_rows<T, TM, NN>(pv, a.ld_dv, t.row0, t.len, a.D, dv, fv);
}

// Blocks 0 .. slots Hkv - 1 own key tiles (from the first one on: in a causal
// sequence the one that most rows see), the others query tiles (from the last
// one back).
template <typename T, int BT, int DMAX>
__global__ void __launch_bounds__(kThreads) attn_bwd_generic(const AttnArgs a, int slots) {
  extern __shared__ float sm[];
  pdl_wait();
  pdl_trigger();
  if (attn_skipped(a.skip)) return;
  const int keys = slots * a.Hkv, b = (int)blockIdx.x;
  if (b < keys)
    dkv_tile<T, BT, DMAX>(a, sm, b % a.Hkv, b / a.Hkv);
  else
    dq_tile<T, BT, DMAX>(a, sm, (b - keys) % a.Hq, slots - 1 - (b - keys) / a.Hq);
}

template <typename T, int BT, int DMAX> struct Generic {
  static size_t smem(const AttnArgs &a, int bufs, int tiles) {
    const int ld = ((a.D + 3) & ~3) + 4;
    return (size_t)(bufs * BT * ld + tiles * BT * (BT + 4) + 2 * BT) * sizeof(float);
  }
  static int slots(const AttnArgs &a) { return (int)(a.T / BT + a.B); }

  static cudaError_t fwd(const AttnArgs &a, const DeviceInfo &dev, cudaStream_t s) {
    const size_t n = smem(a, 3, 1);
    blocks_per_sm((const void *)attn_fwd_generic<T, BT, DMAX>, kThreads, n, dev, 1);  // lifts the limit
    return launch_pdl(attn_fwd_generic<T, BT, DMAX>, dim3((unsigned)slots(a) * (unsigned)a.Hq),
                      dim3(kThreads), n, s, a, slots(a));
  }
  static cudaError_t bwd(const AttnArgs &a, const DeviceInfo &dev, cudaStream_t s) {
    const size_t n = smem(a, 4, 2);
    blocks_per_sm((const void *)attn_bwd_generic<T, BT, DMAX>, kThreads, n, dev, 1);
    return launch_pdl(attn_bwd_generic<T, BT, DMAX>,
                      dim3((unsigned)slots(a) * (unsigned)(a.Hq + a.Hkv)), dim3(kThreads), n, s, a,
                      slots(a));
  }
};

// 64-row tiles while four of them fit beside the score tiles (D <= 128), 32-row
// tiles for the larger heads, and for calls whose 64-row tiles would leave SMs
// without one.  Measured, fp32, 4/2 heads of 64, one sequence, 64 rows against 32,
// us: 300 tokens 44, 40 forward and 132, 117 backward; 1,200 tokens 144, 135 and
// 484, 456; 2,400 tokens 281, 310 and 961, 1,014; 4,096 tokens, 32/8 x 128: 5,460,
// 5,920 and 17,230, 21,280.
bool small_tiles(const AttnArgs &a, const DeviceInfo &dev) {
  return a.D > 128 || (a.T / 64 + a.B) * a.Hq < dev.sms;
}

template <typename T>
cudaError_t fwd_of(const AttnArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  if (!small_tiles(a, dev)) return Generic<T, 64, 128>::fwd(a, dev, s);
  return a.D <= 128 ? Generic<T, 32, 128>::fwd(a, dev, s) : Generic<T, 32, 256>::fwd(a, dev, s);
}
template <typename T>
cudaError_t bwd_of(const AttnArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  if (!small_tiles(a, dev)) return Generic<T, 64, 128>::bwd(a, dev, s);
  return a.D <= 128 ? Generic<T, 32, 128>::bwd(a, dev, s) : Generic<T, 32, 256>::bwd(a, dev, s);
}

}  // namespace

cudaError_t launch_attn_fwd_generic(DType dt, const AttnArgs &a, const DeviceInfo &dev,
                                    cudaStream_t s) {
  return dt == DType::F32 ? fwd_of<float>(a, dev, s) : fwd_of<bf16>(a, dev, s);
}

cudaError_t launch_attn_bwd_generic(DType dt, const AttnArgs &a, const DeviceInfo &dev,
                                    cudaStream_t s) {
  return dt == DType::F32 ? bwd_of<float>(a, dev, s) : bwd_of<bf16>(a, dev, s);
}

}  // namespace ftk
