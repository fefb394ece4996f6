// Forward of the joint of a block's output with the residual stream (block_norm.cuh).
//
// Bound by memory: x and res read once, h and y written once, 4 es bytes a column.  The
// two norms follow one another (the second is of the stored h), so that a row meets two
// barriers; two CTAs an SM and two rows at a time fill the waits.  What remains is the
// random numbers' integer work: about 290 instructions a packet of eight columns with
// dropout.  65,536 x 4,096 bf16 with post-norm and dropout: 331 us, 6,480 GB/s, 0.97 of
// the copy rate (three walks of a CTA over its row: 1,045 us; two rows at a time instead
// of one 484 -> 414, two CTAs of 64 registers instead of one of 96 406 -> 353, addresses
// in uniform registers and no branches for the row's end 353 -> 331).
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

// Rows of up to kMaxWarps warps: a persistent grid, W warps a row, B rows at a time (which
// share the weights in registers, the barriers and the shuffles), the rows ahead on
// their way while the group works on the current ones.
template <int N, int V, int WARPS> constexpr int kFwdRows =
    (N > 1 && (V == 1 || (V == 2 && WARPS <= 16))) || (N == 1 && V == 4 && WARPS <= 16) ? 2 : 1;
// rows in the ring, the current ones among them: two turns
template <int N, int V, int WARPS> constexpr int kFwdDepth = 2 * kFwdRows<N, V, WARPS>;

// Up to WARPS warps a CTA, CTAS of them an SM; see fwd_packets for the choice.
template <typename T, int N, int V, bool DROP, int WARPS, int CTAS>
__global__ void __launch_bounds__(32 * WARPS, CTAS)
block_norm_fwd_rows(const BlockNorm<T> a, const Walk<2> walk_in, const Walk<2> walk_out, int W,
                    int R) {
  using VT = typename Values<N>::V;
  using Rw = typename Raw<T, N>::type;
  constexpr int P = Values<N>::kCount, B = kFwdRows<N, V, WARPS>;
  // the weights in registers; else read for each row
  constexpr bool kHold = V * N <= 8 || (V == 2 && WARPS <= 16);
  extern __shared__ uint4 ring[];
  __shared__ float slots[kMaxGroups][2][2][B * kMaxWarps];  // group, parity, which sum
  pdl_wait();
  pdl_trigger();
  const Philox g = philox_of(a.drop);
  const auto [grp, wig, gi, G] = place_of(W);
  auto &sums = slots[W > 1 ? grp : 0];  // rows of one warp need none
  const int c0 = gi * N;
  uint32_t on = 0;
#pragma unroll
  for (int k = 0; k < V; ++k) on |= (gi + k * G) * N < a.H ? 1u << k : 0u;
  VT wg[kHold ? V : 1][P], w[kHold ? V : 1][P];
  if constexpr (kHold)
#pragma unroll
    for (int k = 0; k < V; ++k) {
#pragma unroll
      for (int i = 0; i < P; ++i) wg[k][i] = w[k][i] = vall<VT>(0.f);
      if (on >> k & 1) {
        column_factors<T, N>(a, c0 + k * G * N, wg[k]);
        unpack(load_raw<Rw>(a.w + c0 + k * G * N), w[k]);
      }
    }
  Mask<N, V> mask;
  if (DROP) mask.init(g, a.drop.thr, gi, G);
  const uint32_t rows = (uint32_t)a.rows, step = gridDim.x * R;
  uint32_t t = blockIdx.x * R + grp;
  Rows<2> src{{(const char *)(a.x + t * a.ldx), (const char *)(a.res + t * a.ldr)}};
  Rows<2> dst{{(const char *)(a.h + t * a.ldh), (const char *)(a.y + t * a.ldy)}};
  const uint32_t off = V > 1 || on ? c0 * (int)sizeof(T) : 0, gap = G * N * (int)sizeof(T);
  Turn turn{t, step, rows, off, gap, on};
  Ahead<T, N, V, 2, B, kFwdDepth<N, V, WARPS>> in;
  in.start(ring, src, walk_in, turn);
  float tok[B];
  auto gates = [&](uint32_t n) {
#pragma unroll
    for (int b = 0; b < B; ++b)
      tok[b] = a.gate_tok != nullptr && n + b * step < rows ? a.gate_tok[n + b * step] : 1.f;
  };
  gates(t);
  const VT rs = vall<VT>(a.res_scale);
  const float xs = a.x_scale * a.drop.scale;
  for (int parity = 0; t < rows; t += B * step, parity ^= 1, in.next()) {  // group-uniform
    float f[B], s[B];
#pragma unroll
    for (int b = 0; b < B; ++b) f[b] = tok[b] * xs;
    if (a.gate_tok != nullptr) gates(t + B * step);
    typename Mask<N, V>::Row m[B];
    if (DROP)
#pragma unroll
      for (int b = 0; b < B; ++b) mask.row(g, t + b * step, gi, G, m[b]);
    in.arrive(src, walk_in, turn);
    if (a.w_post != nullptr) {
#pragma unroll
      for (int b = 0; b < B; ++b) {
        VT ss = vall<VT>(0.f);
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (V == 1 || on >> k & 1) {
            VT x[P];
            unpack(in.get(0, b, k), x);
#pragma unroll
            for (int i = 0; i < P; ++i) ss = vfma(x[i], x[i], ss);
          }
        s[b] = V > 1 || on ? vsum(ss) : 0.f;
      }
      group_sums<B>(s, sums[parity][0], W, wig, grp);
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const float r1 = rsqrtf(fmaf(s[b], a.inv_h, a.eps));
        if (a.rstd_post != nullptr && gi == 0 && t + b * step < rows)
          a.rstd_post[t + b * step] = r1;
        f[b] *= r1;
      }
    }
    Rw h[B][V];
    const char *hr = dst.at[0];
#pragma unroll
    for (int b = 0; b < B; ++b, hr += walk_out.step[0]) {
      VT ss = vall<VT>(0.f);
      const VT fv = vall<VT>(f[b]);
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (V == 1 || on >> k & 1) {
          VT x[P], o[P], fk[P];
          unpack(in.get(0, b, k), x);
          unpack(in.get(1, b, k), o);
          if constexpr (!kHold) column_factors<T, N>(a, c0 + k * G * N, fk);
#pragma unroll
          for (int i = 0; i < P; ++i) {
            VT v = vmul(vmul(x[i], fv), kHold ? wg[kHold ? k : 0][i] : fk[i]);
            if (DROP) v = mask.keep(m[b], k, i, v);
            o[i] = vfma(rs, o[i], v);
          }
          pack(o, h[b][k]);
          unpack(h[b][k], o);
#pragma unroll
          for (int i = 0; i < P; ++i) ss = vfma(o[i], o[i], ss);
          if ((on >> k & 1) && (b == 0 || t + b * step < rows))
            store_raw((T *)(hr + (off + k * gap)), h[b][k]);
        }
      s[b] = V > 1 || on ? vsum(ss) : 0.f;
    }
    group_sums<B>(s, sums[parity][1], W, wig, grp);
#pragma unroll
    for (int b = 0; b < B; ++b) {
      if (b > 0 && t + b * step >= rows) break;
      const float r2 = rsqrtf(fmaf(s[b], a.inv_h, a.eps));
      if (a.rstd != nullptr && gi == 0) a.rstd[t + b * step] = r2;
      const VT r2v = vall<VT>(r2);
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (on >> k & 1) {
          VT o[P], fk[P];
          unpack(h[b][k], o);
          if constexpr (!kHold) unpack(load_raw<Rw>(a.w + c0 + k * G * N), fk);
#pragma unroll
          for (int i = 0; i < P; ++i)
            o[i] = vmul(vmul(o[i], r2v), kHold ? w[kHold ? k : 0][i] : fk[i]);
          Rw y;
          pack(o, y);
          store_raw((T *)(dst.at[1] + (off + k * gap)), y);
        }
      dst.advance(walk_out);
    }
    if (B > 1 && t + step >= rows) break;  // the last turn may be short
  }
  cp_async_wait<0>();
}

template <typename T, int N, int V, int WARPS, int CTAS, int CTAS_DROP = CTAS>
cudaError_t fwd_rows(const BlockPlan &p, const BlockNormArgs &a, const DeviceInfo &dev,
                     cudaStream_t s) {
  auto kern = a.drop.thr > 0 ? block_norm_fwd_rows<T, N, V, true, WARPS, CTAS_DROP>
                             : block_norm_fwd_rows<T, N, V, false, WARPS, CTAS>;
  const size_t smem =
      Ahead<T, N, V, 2, kFwdRows<N, V, WARPS>, kFwdDepth<N, V, WARPS>>::bytes(p.threads());
  const int occ = blocks_per_sm((const void *)kern, p.threads(), smem, dev, 8);
  int64_t grid = ceil_div(a.T, (int64_t)p.R);
  if (grid > (int64_t)dev.sms * occ) grid = (int64_t)dev.sms * occ;
  const int64_t step = grid * p.R * (int64_t)sizeof(T);
  return launch_pdl(kern, dim3((unsigned)grid), dim3(p.threads()), smem, s,
                    block_norm_params<T>(a), Walk<2>{{step * a.ldx, step * a.ldr}},
                    Walk<2>{{step * a.ldh, step * a.ldy}}, p.W, p.R);
}

template <typename T>
cudaError_t fwd_any(const BlockNormArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  const int64_t grid = a.T < (int64_t)dev.sms * 8 ? a.T : (int64_t)dev.sms * 8;
  return launch_pdl(block_norm_fwd_any<T>, dim3((unsigned)grid), dim3(kThreads), 0, s,
                    block_norm_params<T>(a));
}

// Rows of whole packets, by the warps that they take with one packet a thread; with
// dropout, measured with the other choices:
//   up to 16  one packet, two CTAs of 64 registers (65,536 x 4,096: 331 us; one CTA 405).
//             Without dropout two and one: 16,384 x 896 19.6 and 22.2 us, 32,768 x 3,200 139
//             and 149, but 65,536 x 2,048 189 and 166, 65,536 x 4,096 366 and 342
//   up to 20  two packets, half the warps: two CTAs of 96 registers (32,768 x 5,120: 211
//             us; one packet and one CTA 243), or without dropout one (207; two 232)
//   up to 32  two packets, one CTA of 128 registers (16,384 x 8,192: 166 us; one row at a
//             time in two CTAs of 64 registers 200)
// then two and four packets with the weights read for each row.  fp32, with half the
// arithmetic for the bytes, always has one CTA (32,768 x 2,048: 172 us, two 184; 32,768 x
// 2,560: 202, two 233).
template <typename T>
cudaError_t fwd_packets(const BlockNormArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  constexpr int N = VecWidth<T>::value, kTwo = sizeof(T) == 2 ? 2 : 1;
  BlockPlan p = plan_block_row(a.H, N, 16);
  if (p.V == 1 && p.W > 16) p = BlockPlan{2, (p.W + 1) / 2, 1};
  switch (p.V) {
    case 1: return fwd_rows<T, N, 1, 16, kTwo>(p, a, dev, s);
    case 2:
      if (p.W <= 10) return fwd_rows<T, N, 2, 10, 1, kTwo>(p, a, dev, s);
      if (p.W <= 16) return fwd_rows<T, N, 2, 16, 1>(p, a, dev, s);
      return fwd_rows<T, N, 2, kMaxWarps, 1>(p, a, dev, s);
    case 4: return fwd_rows<T, N, 4, kMaxWarps, 1>(p, a, dev, s);
    default: return fwd_any<T>(a, dev, s);
  }
}

// Rows of single columns.  Up to 2,048: two rows at a time in one CTA (32,767 x 1,001 bf16:
// 113 us; in two CTAs 123, one row at a time in two 137).
template <typename T>
cudaError_t fwd_columns(const BlockNormArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  const BlockPlan p = plan_block_row(a.H, 1, 16);
  switch (p.V) {
    case 1: return fwd_rows<T, 1, 1, 16, 2>(p, a, dev, s);
    case 4:
      if (p.threads() <= 512) return fwd_rows<T, 1, 4, 16, 1>(p, a, dev, s);
      return fwd_rows<T, 1, 4, kMaxWarps, 1>(p, a, dev, s);
    case 8: return fwd_rows<T, 1, 8, kMaxWarps, 1>(p, a, dev, s);
    default: return fwd_any<T>(a, dev, s);
  }
}

template <typename T>
cudaError_t fwd_typed(bool vec, const BlockNormArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  cudaError_t e = vec ? fwd_packets<T>(a, dev, s) : fwd_columns<T>(a, dev, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_norm_fwd(DType dt, bool vec, const BlockNormArgs &a,
                                  const DeviceInfo &dev, cudaStream_t s) {
  return dt == DType::F32 ? fwd_typed<float>(vec, a, dev, s) : fwd_typed<bf16>(vec, a, dev, s);
}

}  // namespace ftk
