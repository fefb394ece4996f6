// Forward of the joint of a block's output with the residual stream (block_norm.cuh).
#include "block_norm.cuh"

namespace ftk {

namespace {

constexpr int kThreads = 256;

// Rows of any length and alignment: a CTA walks one row at a time, three times.
template <typename T>
__global__ void __launch_bounds__(kThreads) block_norm_fwd_any(const BlockNorm<T> a) {
  __shared__ float red[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const Philox g = philox_of(a.drop);
  for (int64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
    const T *xr = a.x + t * a.ldx, *rr = a.res + t * a.ldr;
    T *hr = a.h + t * a.ldh, *yr = a.y + t * a.ldy;
    float r1 = 1.f;
    if (a.w_post != nullptr) {
      float ss = 0.f;
      for (int j = threadIdx.x; j < a.H; j += kThreads) {
        const float v = to_float(xr[j]);
        ss = fmaf(v, v, ss);
      }
      r1 = rsqrtf(fmaf(cta_sum(ss, red, kThreads / 32), a.inv_h, a.eps));
      if (a.rstd_post != nullptr && threadIdx.x == 0) a.rstd_post[t] = r1;
    }
    const float c = (a.gate_tok != nullptr ? a.gate_tok[t] * a.x_scale : a.x_scale) * a.drop.scale;
    float ss = 0.f;
    for_columns(g, a.drop.thr, t, a.H, [&](int j, bool kept) {
      const float b = kept ? to_float(xr[j]) * r1 * column_factor(a, j) * c : 0.f;
      const T h = from_float<T>(fmaf(a.res_scale, to_float(rr[j]), b));
      hr[j] = h;
      ss = fmaf(to_float(h), to_float(h), ss);
    });
    const float r2 = rsqrtf(fmaf(cta_sum(ss, red, kThreads / 32), a.inv_h, a.eps));
    if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[t] = r2;
    for_columns(g, 0, t, a.H, [&](int j, bool) {  // the columns that this thread wrote
      yr[j] = from_float<T>(to_float(hr[j]) * r2 * to_float(a.w[j]));
    });
  }
}

// Rows of up to kMaxWarps warps: a persistent grid, W warps a row, the rows ahead on
// their way while the group works on the current one.
// rows in the ring, the current one among them (four packets a thread leave room for two)
template <int V> constexpr int kFwdDepth = V > 2 ? 2 : 3;

constexpr int kFwdWarps = 16, kFwdFirst = 8;

template <typename T, int N, int V, bool DROP>
__global__ void __launch_bounds__(32 * kFwdWarps, 2)
block_norm_fwd_rows(const BlockNorm<T> a, int W, int R) {
  using VT = typename Values<N>::V;
  using Rw = typename Raw<T, N>::type;
  constexpr int P = Values<N>::kCount;
  constexpr bool kHold = V * N <= 8;  // the weights in registers; else read for each row
  extern __shared__ uint4 ring[];
  __shared__ __align__(16) float slots[8][2][2][kMaxWarps + 4];  // group, parity, which sum
  for (int i = threadIdx.x; i < 8 * 4 * (kMaxWarps + 4); i += blockDim.x)
    (&slots[0][0][0][0])[i] = 0.f;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const Philox g = philox_of(a.drop);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = warp / W, wig = warp - grp * W, gi = wig * 32 + lane, G = W * 32;
  const int hp = a.H / N;
  auto col = [&](int k) { return gi + k * G < hp ? (gi + k * G) * N : -1; };
  VT wg[kHold ? V : 1][P];
  Rw w[kHold ? V : 1];
  if constexpr (kHold)
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (col(k) >= 0) {
        column_factors<T, N>(a, col(k), wg[k]);
        w[k] = load_raw<Rw>(a.w + col(k));
      }
  Mask<N, V> mask;
  if (DROP) mask.init(g, a.drop.thr, gi, G);
  const int64_t step = (int64_t)gridDim.x * R;
  auto row = [&](int b, int64_t t) { return b == 0 ? a.x + t * a.ldx : a.res + t * a.ldr; };
  Ahead<T, N, V, 2, kFwdDepth<V>> in;
  in.init(ring);
  int64_t t = (int64_t)blockIdx.x * R + grp;
  in.start(t, step, a.rows, row, col);
  float tok_next = a.gate_tok != nullptr && t < a.rows ? a.gate_tok[t] : 1.f;
  const VT rs = vall<VT>(a.res_scale);
  for (int parity = 0; t < a.rows; t += step, parity ^= 1, in.next()) {  // uniform in the group
    const float c0 = tok_next * a.x_scale * a.drop.scale;
    if (a.gate_tok != nullptr && t + step < a.rows) tok_next = a.gate_tok[t + step];
    if (DROP) mask.row(g, (uint32_t)t, gi, G);
    in.arrive(t, step, a.rows, row, col);
    float r1 = 1.f;
    if (a.w_post != nullptr) {
      VT ss = vall<VT>(0.f);
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (col(k) >= 0) {
          VT x[P];
          unpack(in.get(0, k), x);
#pragma unroll
          for (int i = 0; i < P; ++i) ss = vfma(x[i], x[i], ss);
        }
      r1 = rsqrtf(fmaf(group_sum(vsum(ss), slots[grp][parity][0], W, wig, grp), a.inv_h, a.eps));
      if (a.rstd_post != nullptr && gi == 0) a.rstd_post[t] = r1;
    }
    VT ss = vall<VT>(0.f);
    const VT r1v = vall<VT>(r1), c0v = vall<VT>(c0);
    Rw h[V];
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (col(k) >= 0) {
        VT x[P], f[P], o[P];
        unpack(in.get(0, k), x);
        unpack(in.get(1, k), o);
        if constexpr (!kHold) column_factors<T, N>(a, col(k), f);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          VT b = vmul(vmul(vmul(x[i], r1v), kHold ? wg[kHold ? k : 0][i] : f[i]), c0v);
          if (DROP) b = mask.keep(k, i, b);
          o[i] = vfma(rs, o[i], b);
        }
        pack(o, h[k]);
        store_raw(a.h + t * a.ldh + col(k), h[k]);
        unpack(h[k], o);
#pragma unroll
        for (int i = 0; i < P; ++i) ss = vfma(o[i], o[i], ss);
      }
    const float r2 =
        rsqrtf(fmaf(group_sum(vsum(ss), slots[grp][parity][1], W, wig, grp), a.inv_h, a.eps));
    if (a.rstd != nullptr && gi == 0) a.rstd[t] = r2;
    const VT r2v = vall<VT>(r2);
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (col(k) >= 0) {
        VT o[P], f[P];
        unpack(h[k], o);
        unpack(kHold ? w[kHold ? k : 0] : load_raw<Rw>(a.w + col(k)), f);
#pragma unroll
        for (int i = 0; i < P; ++i) o[i] = vmul(vmul(o[i], r2v), f[i]);
        Rw y;
        pack(o, y);
        store_raw(a.y + t * a.ldy + col(k), y);
      }
  }
}

template <typename T, int N, int V>
cudaError_t fwd_rows(const BlockPlan &p, const BlockNormArgs &a, const DeviceInfo &dev,
                     cudaStream_t s) {
  auto kern = a.drop.thr > 0 ? block_norm_fwd_rows<T, N, V, true>
                             : block_norm_fwd_rows<T, N, V, false>;
  const size_t smem = Ahead<T, N, V, 2, kFwdDepth<V>>::bytes(p.threads());
  const int occ = blocks_per_sm((const void *)kern, p.threads(), smem, dev, 8);
  int64_t grid = ceil_div(a.T, (int64_t)p.R);
  if (grid > (int64_t)dev.sms * occ) grid = (int64_t)dev.sms * occ;
  return launch_pdl(kern, dim3((unsigned)grid), dim3(p.threads()), smem, s,
                    block_norm_params<T>(a), p.W, p.R);
}

template <typename T, int N>
cudaError_t fwd_packets(const BlockNormArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  const BlockPlan p = plan_block_row(a.H / N, N == 1 ? 8 : 4, kFwdFirst, kFwdWarps);
  switch (p.V) {
    case 1: return fwd_rows<T, N, 1>(p, a, dev, s);
    case 2: return fwd_rows<T, N, 2>(p, a, dev, s);
    case 4: return fwd_rows<T, N, 4>(p, a, dev, s);
    case 8:
      if constexpr (N == 1) return fwd_rows<T, N, 8>(p, a, dev, s);
    default: break;
  }
  int64_t grid = a.T < (int64_t)dev.sms * 8 ? a.T : (int64_t)dev.sms * 8;
  return launch_pdl(block_norm_fwd_any<T>, dim3((unsigned)grid), dim3(kThreads), 0, s,
                    block_norm_params<T>(a));
}

template <typename T>
cudaError_t fwd_typed(bool vec, const BlockNormArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  cudaError_t e = vec ? fwd_packets<T, VecWidth<T>::value>(a, dev, s) : fwd_packets<T, 1>(a, dev, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_norm_fwd(DType dt, bool vec, const BlockNormArgs &a,
                                  const DeviceInfo &dev, cudaStream_t s) {
  return dt == DType::F32 ? fwd_typed<float>(vec, a, dev, s) : fwd_typed<bf16>(vec, a, dev, s);
}

}  // namespace ftk
