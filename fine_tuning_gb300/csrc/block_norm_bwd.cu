// Backward of the joint of a block's output with the residual stream (block_norm.cuh).
// With xn = x r1, hn = h r2, wg = w_post gate, m the dropout's mask and
// beta = x_scale / (probability of being kept):
//   G    = dh + r2 w dy - k hn,     k = r2 / H sum_j w dy hn
//   dres = res_scale G
//   c    = beta gate_tok sum_j m wg xn G
//   dx   = r1 (beta gate_tok m wg G) - (r1 / H) c xn        (no second term without w_post)
//   dw   = sum_t dy hn,   S = sum_t beta gate_tok m G xn,   dw_post = gate S, dgate = w_post S
//   dgate_tok[t] = c / gate_tok, formed without the division
// Both row sums come from one pass over the row: with q = m wg xn,
//   sum q G = sum q (dh + r2 w dy) - k sum q hn.
// No product of two r is formed where it may overflow, for rows near zero: each r multiplies
// an h, an x or a sum of them, which it brings back to the size of one.
//
// A CTA's column sums go to its own row of the workspace; a second kernel adds the
// rows in a fixed order and applies gate and w_post.
//
// Memory bound by its bytes (four tensors read, two written, 6 es a column), and in fact
// close to the SM's issue rate with dropout: 400 to 460 instructions a packet of eight
// columns.  What helped was what gives a warp independent work: two rows at a time
// (65,536 x 5,120: 1,146 us with one, 716 with two; in an earlier form 797 with three beside
// 705), and registers: one CTA an SM of 16 warps with 128 registers a thread takes 264 us
// for 32,768 x 4,096 (0.91 of the copy rate), with 96 327, in an earlier form two CTAs with
// 64 334.  Rows of 20 warps have 96: 65,536 x 5,120 716 to 725 us on several GPUs, 5,600
// GB/s, 0.84; 32,768 x 4,608 348, 0.78.  Wider rows take two packets a thread and one row
// at a time, for lack of registers: 16,384 x 8,192 333 us, 0.72; 32,768 x 5,376 527, 0.60.
// Without dropout: 16,384 x 896 32 us (0.82; with it 38.4, 0.68), 32,768 x 4,096 244 (0.99),
// 65,536 x 5,120 650 (0.93), 16,384 x 8,192 298 (0.81), 32,768 x 5,376 468 (0.68).  fp32 with
// dropout: 32,768 x 2,048 243 us (0.99), 32,768 x 4,096 (two packets a thread) 583 (0.83).
// Measured in earlier forms and left: the columns' sums in shared memory 739 against 721;
// ten warps with two packets a thread and two rows 743; the first pass of the next row
// before the second of this one 1,188 against 760.
//
// Spills (bytes a thread, -Xptxas -v): bf16 by four packets a thread with dropout 156 with 16
// warps and 412 with 20, without 0 and 108; by two packets with 20 warps 52 and 16; single
// columns by eight with 20 warps 336 and up to 152; fp32 by four packets with dropout 16.
#include <cfloat>

#include "block_norm.cuh"

namespace ftk {

namespace {

constexpr int kThreads = 512;
constexpr int kMaxBlocksPerSm = 2;  // each has its row of the workspace

// Rows of any length and alignment: a CTA walks one row at a time, twice (4,095 x 5,131
// bf16: 265 us, 950 GB/s).
template <typename T>
__global__ void __launch_bounds__(kThreads, kMaxBlocksPerSm)
block_norm_bwd_any(const BlockNorm<T> a) {
  __shared__ float red[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const Philox g = philox_of(a.drop);
  float *const sum_w = a.ws + (int64_t)blockIdx.x * 2 * a.H, *const sum_s = sum_w + a.H;
  for_columns(g, 0, 0, a.H, [&](int j, bool) { sum_w[j] = sum_s[j] = 0.f; });
  const float beta = a.x_scale * a.drop.scale;
  for (int64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
    const T *xr = a.x + t * a.ldx, *hr = a.h + t * a.ldh;
    const T *gy = a.dy + t * a.lddy, *gh = a.dh + t * a.lddh;
    const float r1 = a.w_post != nullptr ? a.rstd_post[t] : 1.f, r2 = a.rstd[t];
    const float gt = a.gate_tok != nullptr ? a.gate_tok[t] : 1.f;
    float s_h = 0.f, s_g = 0.f, s_c = 0.f;  // sum w dy hn, sum q (dh + r2 w dy), sum q hn
    for_columns(g, a.drop.thr, t, a.H, [&](int j, bool kept) {
      const float wd = to_float(a.w[j]) * to_float(gy[j]), hn = to_float(hr[j]) * r2;
      const float q = kept ? column_factor(a, j) * (to_float(xr[j]) * r1) : 0.f;
      s_h = fmaf(wd, hn, s_h);
      s_g = fmaf(q, fmaf(r2, wd, to_float(gh[j])), s_g);
      s_c = fmaf(q, hn, s_c);
    });
    s_h = cta_sum(s_h, red, kThreads / 32);
    s_g = cta_sum(s_g, red, kThreads / 32);
    s_c = cta_sum(s_c, red, kThreads / 32);
    const float k = r2 * (s_h * a.inv_h);
    const float c = beta * fmaf(-k, s_c, s_g);
    if (a.dgate_tok != nullptr && threadIdx.x == 0) a.dgate_tok[t] = c;
    const float am = a.w_post != nullptr ? r1 * (gt * c * a.inv_h) : 0.f;
    const float bg = beta * gt;
    for_columns(g, a.drop.thr, t, a.H, [&](int j, bool kept) {
      const float dyf = to_float(gy[j]), hn = to_float(hr[j]) * r2;
      // without w_post what is dropped may hold anything
      const float xn = kept || a.w_post != nullptr ? to_float(xr[j]) * r1 : 0.f;
      const float G = fmaf(-k, hn, fmaf(r2, to_float(a.w[j]) * dyf, to_float(gh[j])));
      const float gm = kept ? bg * G : 0.f;
      sum_w[j] = fmaf(dyf, hn, sum_w[j]);
      sum_s[j] = fmaf(gm, xn, sum_s[j]);
      a.dres[t * a.lddr + j] = from_float<T>(a.res_scale * G);
      a.dx[t * a.lddx + j] = from_float<T>(fmaf(-am, xn, r1 * (gm * column_factor(a, j))));
    });
  }
}

// Rows of up to kMaxWarps warps: a persistent grid, W warps a row, B rows at a time (which
// share the weights in registers, the barrier and the shuffles), the rows ahead on their
// way while the group works on the current ones.  Each thread keeps its columns' sums
// for the whole kernel; at the end the CTA's row groups are added in their order.
template <int N, int V> constexpr int kBwdRows = N > 1 && V == 1 ? 2 : 1;
// rows in the ring, the current ones among them: what 227 KB hold
template <int V, int WARPS> constexpr int kBwdDepth =
    V == 1 ? 5 : V == 2 ? (WARPS > 16 ? 2 : 3) : 1;

// One CTA an SM, of up to WARPS warps: 16 (128 registers a thread) or 20 (96), by the
// plan's threads.  Measured, 16 and 20 for rows that 16 hold: 32,768 x 4,096 264 and 327
// us, 65,536 x 2,048 251 and 300, 16,384 x 8,192 333 and 441, 4,095 x 1,001 25.9 and 28.2.
template <typename T, int N, int V, bool DROP, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 1)
block_norm_bwd_rows(const BlockNorm<T> a, const Walk<4> walk_in, const Walk<2> walk_out, int W,
                    int R) {
  using VT = typename Values<N>::V;
  using Rw = typename Raw<T, N>::type;
  constexpr int P = Values<N>::kCount, B = kBwdRows<N, V>;
  // One packet a thread: k r2 and am r1 are one factor each where they fit fp32; where they
  // do not, the row's h and x are multiplied by their r behind a branch, which the whole row
  // takes alike.  Otherwise they always are.  Measured, the branch and the multiplications
  // in every row: 65,536 x 5,120 722 and 784 us, 65,536 x 2,048 251 and 258, but 16,384 x
  // 8,192 340 and 333, 32,767 x 1,001 158 and 155.
  constexpr bool kOneFactor = N > 1 && V == 1;
  // the weights in registers; else read for each row
  constexpr bool kHold = V * N <= (WARPS > 16 ? 8 : 16);
  extern __shared__ uint4 ring[];  // the rows ahead, then [R][2 H] sums when R > 1
  __shared__ float slots[kMaxGroups][2][3 * B * kMaxWarps];  // group, parity
  pdl_wait();
  pdl_trigger();
  const Philox g = philox_of(a.drop);
  const auto [grp, wig, gi, G] = place_of(W);
  auto &sums = slots[W > 1 ? grp : 0];  // rows of one warp need none
  const int c0 = gi * N;
  uint32_t on = 0;
#pragma unroll
  for (int k = 0; k < V; ++k) on |= (gi + k * G) * N < a.H ? 1u << k : 0u;
  VT wg[kHold ? V : 1][P], sw[V][P], sx[V][P];
  Rw w[kHold ? V : 1];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    if constexpr (kHold) {
#pragma unroll
      for (int i = 0; i < P; ++i) wg[k][i] = vall<VT>(0.f);
      w[k] = Rw{};
      if (on >> k & 1) {
        column_factors<T, N>(a, c0 + k * G * N, wg[k]);
        w[k] = load_raw<Rw>(a.w + c0 + k * G * N);
      }
    }
#pragma unroll
    for (int i = 0; i < P; ++i) sw[k][i] = sx[k][i] = vall<VT>(0.f);
  }
  Mask<N, V> mask;
  if (DROP) mask.init(g, a.drop.thr, gi, G);
  const uint32_t rows = (uint32_t)a.rows, step = gridDim.x * R;
  const float beta = a.x_scale * a.drop.scale;
  uint32_t t = blockIdx.x * R + grp;
  Rows<4> src{{(const char *)(a.x + t * a.ldx), (const char *)(a.h + t * a.ldh),
               (const char *)(a.dy + t * a.lddy), (const char *)(a.dh + t * a.lddh)}};
  Rows<2> out{{(const char *)(a.dx + t * a.lddx), (const char *)(a.dres + t * a.lddr)}};
  const uint32_t off = V > 1 || on ? c0 * (int)sizeof(T) : 0, gap = G * N * (int)sizeof(T);
  Turn turn{t, step, rows, off, gap, on};
  Ahead<T, N, V, 4, B, kBwdDepth<V, WARPS>> in;
  in.start(ring, src, walk_in, turn);
  float r1_next[B], r2_next[B], tok_next[B];
  auto scalars = [&](uint32_t n) {
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const bool there = n + b * step < rows;
      r1_next[b] = there && a.w_post != nullptr ? a.rstd_post[n + b * step] : 1.f;
      r2_next[b] = there ? a.rstd[n + b * step] : 0.f;
      tok_next[b] = there && a.gate_tok != nullptr ? a.gate_tok[n + b * step] : 1.f;
    }
  };
  scalars(t);
  for (int parity = 0; t < rows; t += B * step, parity ^= 1, in.next()) {  // group-uniform
    float r1[B], r2[B], gt[B], s[3 * B];
#pragma unroll
    for (int b = 0; b < B; ++b) r1[b] = r1_next[b], r2[b] = r2_next[b], gt[b] = tok_next[b];
    scalars(t + B * step);
    typename Mask<N, V>::Row m[B];
    if (DROP)
#pragma unroll
      for (int b = 0; b < B; ++b) mask.row(g, t + b * step, gi, G, m[b]);
    in.arrive(src, walk_in, turn);
#pragma unroll
    for (int b = 0; b < B; ++b) {
      // without the rows' own factors: w dy h, m wg x (dh + r2 w dy), m wg x h
      VT s_h = vall<VT>(0.f), s_g = s_h, s_c = s_h;
      const VT r2v = vall<VT>(r2[b]);
      if (b == 0 || t + b * step < rows)
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (V == 1 || on >> k & 1) {
            VT x[P], h[P], dy[P], dh[P], f[P], wf[P];
            unpack(in.get(0, b, k), x);
            unpack(in.get(1, b, k), h);
            unpack(in.get(2, b, k), dy);
            unpack(in.get(3, b, k), dh);
            unpack(kHold ? w[kHold ? k : 0] : load_raw<Rw>(a.w + c0 + k * G * N), wf);
            if constexpr (!kHold) column_factors<T, N>(a, c0 + k * G * N, f);
#pragma unroll
            for (int i = 0; i < P; ++i) {
              const VT wd = vmul(wf[i], dy[i]);
              VT q = vmul(kHold ? wg[kHold ? k : 0][i] : f[i], x[i]);
              if (DROP) q = mask.keep(m[b], k, i, q);
              s_h = vfma(wd, h[i], s_h);
              s_g = vfma(q, vfma(r2v, wd, dh[i]), s_g);
              s_c = vfma(q, h[i], s_c);
            }
          }
      const bool mine = V > 1 || on;
      s[3 * b] = mine ? vsum(s_h) : 0.f;
      s[3 * b + 1] = mine ? vsum(s_g) : 0.f;
      s[3 * b + 2] = mine ? vsum(s_c) : 0.f;
    }
    group_sums<3 * B>(s, sums[parity], W, wig, grp);
#pragma unroll
    for (int b = 0; b < B; ++b) {
      if (b > 0 && t + b * step >= rows) break;
      const float kn = r2[b] * (r2[b] * s[3 * b] * a.inv_h);  // k
      const float c1 = beta * (r1[b] * fmaf(-kn, r2[b] * s[3 * b + 2], s[3 * b + 1]));
      if (a.dgate_tok != nullptr && gi == 0) a.dgate_tok[t + b * step] = c1;
      const float am = a.w_post != nullptr ? r1[b] * (gt[b] * c1 * a.inv_h) : 0.f;
      const bool fits = fabsf(kn * r2[b]) <= FLT_MAX && fabsf(am * r1[b]) <= FLT_MAX;
      const bool one = kOneFactor && fits, apart = kOneFactor && !fits;
      const VT r1v = vall<VT>(r1[b]), r2v = vall<VT>(r2[b]), rs = vall<VT>(a.res_scale);
      const VT nk = vall<VT>(one ? -kn * r2[b] : -kn), nam = vall<VT>(one ? -am * r1[b] : -am);
      const VT bg = vall<VT>(beta * gt[b] * r1[b]);
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (V == 1 || on >> k & 1) {
          VT x[P], h[P], dy[P], dh[P], f[P], wf[P];
          unpack(in.get(0, b, k), x);
          unpack(in.get(1, b, k), h);
          unpack(in.get(2, b, k), dy);
          unpack(in.get(3, b, k), dh);
          unpack(kHold ? w[kHold ? k : 0] : load_raw<Rw>(a.w + c0 + k * G * N), wf);
          if constexpr (!kHold) column_factors<T, N>(a, c0 + k * G * N, f);
          if (DROP && a.w_post == nullptr)  // then what is dropped may hold anything
#pragma unroll
            for (int i = 0; i < P; ++i) x[i] = mask.keep(m[b], k, i, x[i]);
#pragma unroll
          for (int i = 0; i < P; ++i) {
            if (kOneFactor) {
              dy[i] = vmul(dy[i], r2v);
              dh[i] = vfma(wf[i], dy[i], dh[i]);
            } else {
              h[i] = vmul(h[i], r2v);
              dh[i] = vfma(r2v, vmul(wf[i], dy[i]), dh[i]);
            }
            sw[k][i] = vfma(dy[i], h[i], sw[k][i]);
          }
          if (apart)
#pragma unroll
            for (int i = 0; i < P; ++i) h[i] = vmul(h[i], r2v);
#pragma unroll
          for (int i = 0; i < P; ++i) {
            const VT Gv = vfma(nk, h[i], dh[i]);
            VT gm = vmul(bg, Gv);  // beta gate_tok r1 m G
            if (DROP) gm = mask.keep(m[b], k, i, gm);
            sx[k][i] = vfma(gm, x[i], sx[k][i]);
            dh[i] = vmul(rs, Gv);
            h[i] = vmul(gm, kHold ? wg[kHold ? k : 0][i] : f[i]);
          }
          if (apart)
#pragma unroll
            for (int i = 0; i < P; ++i) x[i] = vmul(x[i], r1v);
#pragma unroll
          for (int i = 0; i < P; ++i)
            x[i] = vfma(nam, kOneFactor ? x[i] : vmul(x[i], r1v), h[i]);
          Rw oh, ox;
          pack(dh, oh);
          pack(x, ox);
          if (on >> k & 1) {
            store_raw((T *)(out.at[1] + (off + k * gap)), oh);
            store_raw((T *)(out.at[0] + (off + k * gap)), ox);
          }
        }
      out.advance(walk_out);
    }
  }
  cp_async_wait<0>();
  if (R > 1) __syncthreads();  // the ring becomes the row groups' sums
  float *const dst = a.ws + (int64_t)blockIdx.x * 2 * a.H;
  float *const comb = reinterpret_cast<float *>(ring);
  float *const mine = (R > 1 ? comb + grp * 2 * a.H : dst) + c0;
#pragma unroll
  for (int k = 0; k < V; ++k)
    if (on >> k & 1)
#pragma unroll
      for (int i = 0; i < P; ++i) {
        reinterpret_cast<VT *>(mine + k * G * N)[i] = sw[k][i];
        reinterpret_cast<VT *>(mine + a.H + k * G * N)[i] = sx[k][i];
      }
  if (R == 1) return;
  __syncthreads();
  for (int j = threadIdx.x; j < 2 * a.H; j += blockDim.x) {
    float v = comb[j];
    for (int i = 1; i < R; ++i) v += comb[i * 2 * a.H + j];
    dst[j] = v;
  }
}

constexpr int kReduceWarps = 32;
constexpr int kReduceBatch = 5;  // rows of a warp in flight: 160, the sums of one CTA an SM

// dw[j] = sum_p ws[p][j]; S[j] = sum_p ws[p][H + j], dw_post = gate S, dgate = w_post S.
// A CTA owns 32 columns; its warps take the rows p = warp, warp + 32, ... and their
// sums are added in the warps' order.
template <typename T>
__global__ void __launch_bounds__(32 * kReduceWarps)
block_norm_dw(const float *ws, int P, int H, const T *w_post, const T *gate, float *dw,
              float *dw_post, float *dgate) {
  __shared__ float part[kReduceWarps][33];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j = blockIdx.x * 32 + lane;
  const bool shared = blockIdx.y != 0;  // the column sums that dw_post and dgate share
  float s = 0.f;
  if (j < H) {
    const float *col = ws + (shared ? H : 0) + j;
    for (int p0 = warp; p0 < P; p0 += kReduceWarps * kReduceBatch) {
      float v[kReduceBatch];
#pragma unroll
      for (int i = 0; i < kReduceBatch; ++i) {
        const int p = p0 + i * kReduceWarps;
        v[i] = p < P ? __ldcg(col + (int64_t)p * 2 * H) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < kReduceBatch; ++i) s += v[i];
    }
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || j >= H) return;
  float v = 0.f;
#pragma unroll
  for (int i = 0; i < kReduceWarps; ++i) v += part[i][lane];
  if (!shared) {
    dw[j] = v;
    return;
  }
  if (dw_post != nullptr) dw_post[j] = gate != nullptr ? to_float(gate[j]) * v : v;
  if (dgate != nullptr) dgate[j] = w_post != nullptr ? to_float(w_post[j]) * v : v;
}

template <typename T>
cudaError_t reduce(const BlockNormArgs &a, int64_t P, cudaStream_t s) {
  const bool shared = a.dw_post != nullptr || a.dgate != nullptr;
  cudaError_t e = launch_pdl(block_norm_dw<T>,
                             dim3((unsigned)ceil_div(a.H, (int64_t)32), shared ? 2 : 1),
                             dim3(32 * kReduceWarps), 0, s, a.ws, (int)P, (int)a.H,
                             (const T *)a.w_post, (const T *)a.gate, a.dw, a.dw_post, a.dgate);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int N, int V, int WARPS>
cudaError_t bwd_rows(const BlockPlan &p, const BlockNormArgs &a, const DeviceInfo &dev,
                     cudaStream_t s) {
  auto kern = a.drop.thr > 0 ? block_norm_bwd_rows<T, N, V, true, WARPS>
                             : block_norm_bwd_rows<T, N, V, false, WARPS>;
  size_t smem = Ahead<T, N, V, 4, kBwdRows<N, V>, kBwdDepth<V, WARPS>>::bytes(p.threads());
  const size_t sums = p.R > 1 ? (size_t)p.R * 2 * (size_t)a.H * sizeof(float) : 0;
  if (sums > smem) smem = sums;
  const int occ = blocks_per_sm((const void *)kern, p.threads(), smem, dev, kMaxBlocksPerSm);
  int64_t P = ceil_div(a.T, (int64_t)p.R);
  if (P > (int64_t)dev.sms * occ) P = (int64_t)dev.sms * occ;
  const int64_t step = P * p.R * (int64_t)sizeof(T);
  cudaError_t e = launch_pdl(
      kern, dim3((unsigned)P), dim3(p.threads()), smem, s, block_norm_params<T>(a),
      Walk<4>{{step * a.ldx, step * a.ldh, step * a.lddy, step * a.lddh}},
      Walk<2>{{step * a.lddx, step * a.lddr}}, p.W, p.R);
  return e != cudaSuccess ? e : reduce<T>(a, P, s);
}

template <typename T>
cudaError_t bwd_any(const BlockNormArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  const int64_t P = block_norm_partial_rows(a.T, dev);
  cudaError_t e = launch_pdl(block_norm_bwd_any<T>, dim3((unsigned)P), dim3(kThreads), 0, s,
                             block_norm_params<T>(a));
  return e != cudaSuccess ? e : reduce<T>(a, P, s);
}

// The instance with 16 or 20 warps, by the plan's threads.
template <typename T, int N, int V>
cudaError_t bwd_warps(const BlockPlan &p, const BlockNormArgs &a, const DeviceInfo &dev,
                      cudaStream_t s) {
  return p.threads() <= 512 ? bwd_rows<T, N, V, 16>(p, a, dev, s)
                            : bwd_rows<T, N, V, kMaxWarps>(p, a, dev, s);
}

// Rows of whole packets.
template <typename T>
cudaError_t bwd_packets(const BlockNormArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  constexpr int N = VecWidth<T>::value;
  const BlockPlan p = plan_block_row(a.H, N, 16);
  switch (p.V) {
    case 1: return bwd_warps<T, N, 1>(p, a, dev, s);
    case 2: return bwd_warps<T, N, 2>(p, a, dev, s);
    case 4: return bwd_warps<T, N, 4>(p, a, dev, s);
    default: return bwd_any<T>(a, dev, s);
  }
}

// Rows of single columns.
template <typename T>
cudaError_t bwd_columns(const BlockNormArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  const BlockPlan p = plan_block_row(a.H, 1, 16);
  switch (p.V) {
    case 1: return bwd_rows<T, 1, 1, 16>(p, a, dev, s);
    case 4: return bwd_warps<T, 1, 4>(p, a, dev, s);
    case 8: return bwd_warps<T, 1, 8>(p, a, dev, s);
    default: return bwd_any<T>(a, dev, s);
  }
}

template <typename T>
cudaError_t bwd_typed(bool vec, const BlockNormArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  if (a.T == 0) return reduce<T>(a, 0, s);
  return vec ? bwd_packets<T>(a, dev, s) : bwd_columns<T>(a, dev, s);
}

}  // namespace

int64_t block_norm_partial_rows(int64_t T, const DeviceInfo &dev) {
  const int64_t cap = (int64_t)dev.sms * kMaxBlocksPerSm;
  return T < cap ? T : cap;
}

cudaError_t launch_block_norm_bwd(DType dt, bool vec, const BlockNormArgs &a,
                                  const DeviceInfo &dev, cudaStream_t s) {
  return dt == DType::F32 ? bwd_typed<float>(vec, a, dev, s) : bwd_typed<bf16>(vec, a, dev, s);
}

}  // namespace ftk
