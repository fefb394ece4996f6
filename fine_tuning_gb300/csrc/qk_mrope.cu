// Rotary embedding of Q and K by positions on several axes (time, height and
// width, say), rotate-half layout, forward and backward:
//   phi_i(t) = pos[axis_of[i]][t] f_i,  y[i] = x[i] cos - x[i+D/2] sin,
//   y[i+D/2] = x[i+D/2] cos + x[i] sin  (backward: phi -> -phi)
//
// A CTA owns kTok tokens.  It forms each token's D/2 angles once (the
// extended-precision product and sincospi of rope_common.cuh) into a shared
// table of cosines and sines, and then walks the (token, head, packet) units
// of all Q and K heads: one 16-byte packet of each half per thread and unit,
// kUnroll units' loads issued before the first store.  Bound by HBM: 4 bytes
// per element (bf16 in and out); the table costs 64 bytes of shared memory
// per 64 bytes of HBM traffic, a fifth of what the SM can read.
#include "rope_common.cuh"

namespace ftk {

namespace {

constexpr int kMropeThreads = 256;
constexpr int kMropeUnroll = 4;

// What varies by frequency: read by index, so it stays in the constant bank.
struct MropeFreqs {
  RopeFreqs f;
  uint8_t axis[kRopeMaxHalf];
};
struct MropeView {
  const void *in;
  void *out;
  int64_t ld_in, ld_out;
};

// N: values per packet.  half = D/2, nv = half / N packets per half head,
// unit u of the CTA: packet u % nv of head (u / nv) % H of token u / (nv H).
template <typename T, int N>
__global__ void __launch_bounds__(kMropeThreads)
qk_mrope_kernel(const __grid_constant__ MropeFreqs fr, MropeView q, MropeView k,
                const int32_t *__restrict__ pos, int64_t ld_pos, int64_t tokens, int Hq, int H,
                int half, int nv, int tok, float sign) {
  extern __shared__ float tab[];  // cos [tok][half], then sin
  pdl_wait();
  pdl_trigger();
  const int64_t t0 = (int64_t)blockIdx.x * tok;
  const int nt = (int)(tokens - t0 < tok ? tokens - t0 : tok);
  float *cs = tab, *sn = tab + tok * half;
  for (int e = threadIdx.x; e < nt * half; e += kMropeThreads) {
    const int t = e / half, i = e - t * half;
    const int p = __ldg(pos + (int64_t)fr.axis[i] * ld_pos + t0 + t);
    float c, s;
    rope_cos_sin(p, fr.f.hi[i], fr.f.lo[i], &c, &s);
    cs[e] = c;
    sn[e] = sign * s;
  }
  __syncthreads();
  const int D = 2 * half, units = nt * H * nv;
  for (int u0 = threadIdx.x; u0 < units; u0 += kMropeThreads * kMropeUnroll) {
    Packet<T, N> a[kMropeUnroll], b[kMropeUnroll];
    T *dst[kMropeUnroll];
    int at[kMropeUnroll];
#pragma unroll
    for (int n = 0; n < kMropeUnroll; ++n) {
      const int u = u0 + n * kMropeThreads;
      if (u >= units) break;
      const int w = u / nv, j = u - w * nv, t = w / H, h = w - t * H;
      const bool is_q = h < Hq;
      const int hh = is_q ? h : h - Hq;
      const int64_t row = t0 + t;
      const T *src = (const T *)(is_q ? q.in : k.in) + row * (is_q ? q.ld_in : k.ld_in) +
                     (int64_t)hh * D + j * N;
      dst[n] = (T *)(is_q ? q.out : k.out) + row * (is_q ? q.ld_out : k.ld_out) +
               (int64_t)hh * D + j * N;
      at[n] = t * half + j * N;
      a[n] = load_packet_stream<T, N>(src);
      b[n] = load_packet_stream<T, N>(src + half);
    }
#pragma unroll
    for (int n = 0; n < kMropeUnroll; ++n) {
      if (u0 + n * kMropeThreads >= units) break;
      Packet<T, N> ya, yb;
      float va[N], vb[N];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float c = cs[at[n] + e], s = sn[at[n] + e];
        const float x = a[n].get(e), y = b[n].get(e);
        va[e] = x * c - y * s;
        vb[e] = y * c + x * s;
      }
      if constexpr (N == 1) {
        ya.set(0, va[0]);
        yb.set(0, vb[0]);
      } else {
#pragma unroll
        for (int e = 0; e < N; e += 2) {
          ya.set2(e, va[e], va[e + 1]);
          yb.set2(e, vb[e], vb[e + 1]);
        }
      }
      store_packet<T, N>(dst[n], ya);
      store_packet<T, N>(dst[n] + half, yb);
    }
  }
}

template <typename T, int N>
cudaError_t launch(const QkMropeArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  MropeFreqs fr;
  fr.f = make_rope_freqs(a.D, a.theta, a.inv_freq);
  const int half = a.D / 2, nv = half / N, H = a.Hq + a.Hkv;
  for (int i = 0; i < kRopeMaxHalf; ++i) fr.axis[i] = i < half ? (uint8_t)a.axis_of[i] : 0;
  // tokens per CTA: about eight rounds of units, at most 16 tokens
  int tok = (8 * kMropeThreads * N) / (half * H);
  tok = tok < 1 ? 1 : tok > 16 ? 16 : tok;
  const int64_t grid = ceil_div(a.T, (int64_t)tok);
  const MropeView q{a.q, a.oq, a.ld_q, a.ld_oq}, k{a.k, a.ok, a.ld_k, a.ld_ok};
  return launch_pdl(qk_mrope_kernel<T, N>, dim3((unsigned)grid), dim3(kMropeThreads),
                    (size_t)tok * half * 2 * sizeof(float), s, fr, q, k, a.pos, a.ld_pos, a.T, a.Hq,
                    H, half, nv, tok, a.backward ? -1.f : 1.f);
}

}  // namespace

cudaError_t launch_qk_mrope(DType dt, bool vec, const QkMropeArgs &a, const DeviceInfo &dev,
                            cudaStream_t s) {
  if (dt == DType::F32) return vec ? launch<float, 4>(a, dev, s) : launch<float, 1>(a, dev, s);
  return vec ? launch<bf16, 8>(a, dev, s) : launch<bf16, 1>(a, dev, s);
}

}  // namespace ftk
