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
// shared key head are summed over its query heads inside the CTA.  Thread
// (ty, tx) of 16 x 16 holds BT/16 rows x BT/16 columns of the score tile and
// BT/16 rows x D/16 columns of the outputs; operands are read from shared
// memory as float4 along d, rows padded by 4 words so that 8 lanes' float4
// reads fall into different banks.  Bound by shared-memory reads: 2 x 4
// LDS.128 feed 64 multiply-adds.
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

// out[i][n] += sum_c p[ty TM + i][c] b[c][tx + 16 n], c < nc
template <int TM, int NN>
__device__ __forceinline__ void rows_mul(float (&out)[TM][NN], const float *p, int ldp,
                                         const float *b, int ld, int nc, int DP) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int c = 0; c < nc; ++c) {
    float x[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i) x[i] = p[(ty * TM + i) * ldp + c];
#pragma unroll
    for (int n = 0; n < NN; ++n) {
      const int d = tx + 16 * n;
      if (d >= DP) break;
      const float y = b[c * ld + d];
#pragma unroll
      for (int i = 0; i < TM; ++i) out[i][n] = fmaf(x[i], y, out[i][n]);
    }
  }
}

template <typename T, int TM, int NN>
__device__ __forceinline__ void store_rows(T *base, int64_t stride, int row0, int len, int D,
                                           const float (&out)[TM][NN], const float (&f)[TM]) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int r = row0 + ty * TM + i;
    if (r >= len) continue;
    T *p = base + (int64_t)r * stride;
#pragma unroll
    for (int n = 0; n < NN; ++n)
      if (tx + 16 * n < D) p[tx + 16 * n] = from_float<T>(out[i][n] * f[i]);
  }
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

template <typename T, int BT, int DMAX>
__global__ void __launch_bounds__(kThreads)
attn_fwd_generic(const AttnArgs a, int slots) {
  constexpr int TM = BT / 16, NN = DMAX / 16, LDP = BT + 4;
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
  float out[TM][NN], m[TM], l[TM];
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int n = 0; n < NN; ++n) out[i][n] = 0.f;
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
      mx = row_max(mx);  // key 0 is seen by every row: finite from the first tile on
      const float f = expf(m[i] - mx);
      m[i] = mx;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const float p = expf(s[i][j] - mx);
        sum += p;
        Ps[(ty * TM + i) * LDP + tx + 16 * j] = p;
      }
      l[i] = l[i] * f + row_sum(sum);
#pragma unroll
      for (int n = 0; n < NN; ++n) out[i][n] *= f;
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

// delta[h, t] = sum_d do[t, h, d] o[t, h, d]: a warp per (token, head).
template <typename T>
__global__ void __launch_bounds__(kThreads) attn_delta_generic(const AttnArgs a) {
  pdl_wait();
  pdl_trigger();
  if (attn_skipped(a.skip)) return;
  const int64_t rows = a.T * a.Hq;
  const int lane = threadIdx.x & 31;
  for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < rows;
       i += (int64_t)gridDim.x * (kThreads / 32)) {
    const int64_t t = i / a.Hq;
    const int h = (int)(i - t * a.Hq);
    const T *g = (const T *)a.do_ + t * a.ld_do + (int64_t)h * a.D;
    const T *o = (const T *)a.o + t * a.ld_o + (int64_t)h * a.D;
    float s = 0.f;
    for (int d = lane; d < a.D; d += 32) s = fmaf(to_float(g[d]), to_float(o[d]), s);
    s = warp_sum(s);
    if (lane == 0) a.delta[(int64_t)h * a.T + t] = s;
  }
}

template <typename T, int BT, int DMAX>
__global__ void __launch_bounds__(kThreads)
attn_dq_generic(const AttnArgs a, int slots) {
  constexpr int TM = BT / 16, NN = DMAX / 16, LDP = BT + 4;
  extern __shared__ float sm[];
  pdl_wait();
  pdl_trigger();
  if (attn_skipped(a.skip)) return;
  const int DP = (a.D + 3) & ~3, ld = DP + 4;
  float *Qs = sm, *Gs = Qs + BT * ld, *Ks = Gs + BT * ld, *Vs = Ks + BT * ld, *Ds = Vs + BT * ld;
  const int h = blockIdx.x % a.Hq, slot = slots - 1 - (int)(blockIdx.x / a.Hq);
  const SeqTile t = seq_tile(slot, a.cu, a.B, (int)a.T, BT);
  if (t.len == 0) return;
  const int hk = h / (a.Hq / a.Hkv);
  const T *q = (const T *)a.q + t.start * a.ld_q + (int64_t)h * a.D;
  const T *g = (const T *)a.do_ + t.start * a.ld_do + (int64_t)h * a.D;
  const T *k = (const T *)a.k + t.start * a.ld_k + (int64_t)hk * a.D;
  const T *v = (const T *)a.v + t.start * a.ld_v + (int64_t)hk * a.D;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  load_rows<T, BT>(Qs, ld, q, a.ld_q, t.row0, t.len, a.D, DP);
  load_rows<T, BT>(Gs, ld, g, a.ld_do, t.row0, t.len, a.D, DP);
  float out[TM][NN], lse[TM], delta[TM], f[TM];
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int r = t.row0 + ty * TM + i;
    const int64_t at = (int64_t)h * a.T + t.start + r;
    lse[i] = r < t.len ? a.lse[at] : 0.f;
    delta[i] = r < t.len ? a.delta[at] : 0.f;
    f[i] = a.scale;
#pragma unroll
    for (int n = 0; n < NN; ++n) out[i][n] = 0.f;
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
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const int c = c0 + tx + 16 * j;
        const bool see = c < t.len && r < t.len && (!a.causal || c <= r);
        const float p = see ? expf(fmaf(s[i][j], a.scale, -lse[i])) : 0.f;
        Ds[(ty * TM + i) * LDP + tx + 16 * j] = see ? p * (dp[i][j] - delta[i]) : 0.f;
      }
    }
    __syncthreads();
    rows_mul<TM, NN>(out, Ds, LDP, Ks, ld, min(BT, t.len - c0), DP);
  }
  T *dq = (T *)a.dq + t.start * a.ld_dq + (int64_t)h * a.D;
  store_rows<T, TM, NN>(dq, a.ld_dq, t.row0, t.len, a.D, out, f);
}

// Rows are keys, columns queries: the score tile is transposed.
template <typename T, int BT, int DMAX>
__global__ void __launch_bounds__(kThreads)
attn_dkv_generic(const AttnArgs a) {
  constexpr int TM = BT / 16, NN = DMAX / 16, LDP = BT + 4;
  extern __shared__ float sm[];
  pdl_wait();
  pdl_trigger();
  if (attn_skipped(a.skip)) return;
  const int DP = (a.D + 3) & ~3, ld = DP + 4;
  float *Ks = sm, *Vs = Ks + BT * ld, *Qs = Vs + BT * ld, *Gs = Qs + BT * ld, *Ps = Gs + BT * ld;
  float *Ds = Ps + BT * LDP, *Ls = Ds + BT * LDP, *Dl = Ls + BT;
  const int hk = blockIdx.x % a.Hkv, slot = (int)(blockIdx.x / a.Hkv);
  const SeqTile t = seq_tile(slot, a.cu, a.B, (int)a.T, BT);
  if (t.len == 0) return;
  const int G = a.Hq / a.Hkv;
  const T *k = (const T *)a.k + t.start * a.ld_k + (int64_t)hk * a.D;
  const T *v = (const T *)a.v + t.start * a.ld_v + (int64_t)hk * a.D;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  load_rows<T, BT>(Ks, ld, k, a.ld_k, t.row0, t.len, a.D, DP);
  load_rows<T, BT>(Vs, ld, v, a.ld_v, t.row0, t.len, a.D, DP);
  float dk[TM][NN], dv[TM][NN], fk[TM], fv[TM];
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    fk[i] = a.scale;
    fv[i] = 1.f;
#pragma unroll
    for (int n = 0; n < NN; ++n) dk[i][n] = dv[i][n] = 0.f;
  }
  for (int h = hk * G; h < (hk + 1) * G; ++h) {
    const T *q = (const T *)a.q + t.start * a.ld_q + (int64_t)h * a.D;
    const T *g = (const T *)a.do_ + t.start * a.ld_do + (int64_t)h * a.D;
    for (int c0 = a.causal ? t.row0 : 0; c0 < t.len; c0 += BT) {
      __syncthreads();
      load_rows<T, BT>(Qs, ld, q, a.ld_q, c0, t.len, a.D, DP);
      load_rows<T, BT>(Gs, ld, g, a.ld_do, c0, t.len, a.D, DP);
      if (threadIdx.x < BT) {
        const int c = c0 + threadIdx.x;
        const int64_t at = (int64_t)h * a.T + t.start + c;
        Ls[threadIdx.x] = c < t.len ? a.lse[at] : 0.f;
        Dl[threadIdx.x] = c < t.len ? a.delta[at] : 0.f;
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

template <typename T, int BT, int DMAX> struct Generic {
  static size_t smem(const AttnArgs &a, int bufs, int tiles) {
    const int ld = ((a.D + 3) & ~3) + 4;
    return (size_t)(bufs * BT * ld + tiles * BT * (BT + 4) + 2 * BT) * sizeof(float);
  }
  template <typename K> static cudaError_t prepare(K kern, size_t smem, const DeviceInfo &dev) {
    blocks_per_sm((const void *)kern, kThreads, smem, dev, 1);  // lifts the shared memory limit
    return cudaSuccess;
  }
  static int slots(const AttnArgs &a) { return (int)(a.T / BT + a.B); }

  static cudaError_t fwd(const AttnArgs &a, const DeviceInfo &dev, cudaStream_t s) {
    const size_t n = smem(a, 3, 1);
    cudaError_t e = prepare(attn_fwd_generic<T, BT, DMAX>, n, dev);
    if (e != cudaSuccess) return e;
    return launch_pdl(attn_fwd_generic<T, BT, DMAX>, dim3((unsigned)slots(a) * (unsigned)a.Hq),
                      dim3(kThreads), n, s, a, slots(a));
  }
  static cudaError_t bwd(const AttnArgs &a, const DeviceInfo &dev, cudaStream_t s) {
    size_t n = smem(a, 4, 1);
    cudaError_t e = prepare(attn_dq_generic<T, BT, DMAX>, n, dev);
    if (e != cudaSuccess) return e;
    e = launch_pdl(attn_dq_generic<T, BT, DMAX>, dim3((unsigned)slots(a) * (unsigned)a.Hq),
                   dim3(kThreads), n, s, a, slots(a));
    if (e != cudaSuccess) return e;
    n = smem(a, 4, 2);
    e = prepare(attn_dkv_generic<T, BT, DMAX>, n, dev);
    if (e != cudaSuccess) return e;
    return launch_pdl(attn_dkv_generic<T, BT, DMAX>, dim3((unsigned)slots(a) * (unsigned)a.Hkv),
                      dim3(kThreads), n, s, a);
  }
};

template <typename T> cudaError_t delta_of(const AttnArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  const int64_t want = ceil_div(a.T * a.Hq, (int64_t)(kThreads / 32));
  const int64_t most = (int64_t)dev.sms * 16;
  return launch_pdl(attn_delta_generic<T>, dim3((unsigned)(want < most ? want : most)),
                    dim3(kThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_attn_delta(DType dt, const AttnArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  return dt == DType::F32 ? delta_of<float>(a, dev, s) : delta_of<bf16>(a, dev, s);
}

// 64-row tiles while four of them fit beside the score tiles (D <= 128),
// 32-row tiles for the larger heads.
cudaError_t launch_attn_fwd_generic(DType dt, const AttnArgs &a, const DeviceInfo &dev,
                                    cudaStream_t s) {
  if (dt == DType::F32)
    return a.D <= 128 ? Generic<float, 64, 128>::fwd(a, dev, s)
                      : Generic<float, 32, 256>::fwd(a, dev, s);
  return a.D <= 128 ? Generic<bf16, 64, 128>::fwd(a, dev, s)
                    : Generic<bf16, 32, 256>::fwd(a, dev, s);
}

cudaError_t launch_attn_bwd_generic(DType dt, const AttnArgs &a, const DeviceInfo &dev,
                                    cudaStream_t s) {
  cudaError_t e = launch_attn_delta(dt, a, dev, s);
  if (e != cudaSuccess) return e;
  if (dt == DType::F32)
    return a.D <= 128 ? Generic<float, 64, 128>::bwd(a, dev, s)
                      : Generic<float, 32, 256>::bwd(a, dev, s);
  return a.D <= 128 ? Generic<bf16, 64, 128>::bwd(a, dev, s)
                    : Generic<bf16, 32, 256>::bwd(a, dev, s);
}

}  // namespace ftk
