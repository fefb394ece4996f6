// Rotary embedding of Q and K by positions on several axes (time, height and
// width, say), rotate-half layout, forward and backward:
//   phi_i(t) = pos[axis_of[i]][t] f_i,  y[i] = x[i] cos - x[i+D/2] sin,
//   y[i+D/2] = x[i+D/2] cos + x[i] sin  (backward: phi -> -phi)
//
// A CTA owns tok tokens.  It forms each token's D/2 angles once (the
// extended-precision product and sincospi of rope_common.cuh) into a shared
// table of cosines and sines.  A thread then keeps the cosines and sines of
// one (token, packet) in registers and walks every S-th head of Q and K: one
// 16-byte packet of each half per head, kMropeUnroll heads' loads issued
// before the first store.  Bound by HBM, 4 bytes per element (bf16 in and out):
// 207 us on 65,536 tokens x 32/8 bf16 heads of 128 (6.48 TB/s, 0.96 of the copy
// rate), 100 us on 32,767 tokens x 32/8 fp32 heads of 64 (6.7 TB/s); with few heads
// by the angles: 23 us on 68,158 tokens x 1/1 bf16 heads of 96 (2.3 TB/s).  Measured
// on the way, first call: the table read from shared memory for every head,
// 346 us; in registers with four heads in flight but two CTAs per SM, 345; two
// heads and four CTAs, 266 (bf16 values converted one by one, spilling); pairs,
// 215; frequencies from shared memory instead of the constant bank, 207 (the last
// call: 74 before, 23 after).
#include "launch_attn.h"
#include "pair_math.cuh"
#include "rope_common.cuh"

namespace ftk {

namespace {

constexpr int kMropeThreads = 256;
// heads in flight per thread: with two of 8-value packets (16 registers each,
// beside 16 cosines and sines) four CTAs fit an SM; with four, two
template <int N> constexpr int kMropeUnroll = N == 8 ? 2 : 4;

// What varies by frequency.  A CTA copies it to shared memory first: lanes that
// read 32 different entries of the constant bank are served one by one, which
// for every angle anew costs more than the angles.
struct MropeFreqs {
  RopeFreqs f;
  uint8_t axis[kRopeMaxHalf];
};
struct MropeView {
  const void *in;
  void *out;
  int64_t ld_in, ld_out;
};

// One packet of each half turned by its angles: a <- a c - b s, b <- b c + a s,
// the first product of each rounded, the second fused, in both forms (eight
// bf16 as four fp32 pairs, or value by value), so they give the same bits.
template <typename T, int N>
__device__ __forceinline__ void turn(Packet<T, N> &a, Packet<T, N> &b, const float (&c)[N],
                                     const float (&s)[N]) {
  if constexpr (sizeof(T) == 2 && N == 8) {
    float2 x[4], y[4];
    unpack8(*reinterpret_cast<const uint4 *>(&a), x);
    unpack8(*reinterpret_cast<const uint4 *>(&b), y);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 ce = make_float2(c[2 * e], c[2 * e + 1]);
      const float2 se = make_float2(s[2 * e], s[2 * e + 1]);
      const float2 ys = __fmul2_rn(y[e], se), xs = __fmul2_rn(x[e], se);
      x[e] = __ffma2_rn(x[e], ce, make_float2(-ys.x, -ys.y));
      y[e] = __ffma2_rn(y[e], ce, xs);
    }
    *reinterpret_cast<uint4 *>(&a) = pack8(x);
    *reinterpret_cast<uint4 *>(&b) = pack8(y);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float x = a.get(e), y = b.get(e);
      const float ys = __fmul_rn(y, s[e]), xs = __fmul_rn(x, s[e]);
      a.set(e, fmaf(x, c[e], -ys));
      b.set(e, fmaf(y, c[e], xs));
    }
  }
}

// N: values per packet; half = D/2, nv = half / N packets per half head.
// Thread tid: packet tid % nv, head slot (tid / nv) % S, token tid / (nv S).
template <typename T, int N>
__global__ void __launch_bounds__(kMropeThreads, 4)
qk_mrope_kernel(const __grid_constant__ MropeFreqs fr, MropeView q, MropeView k,
                const int32_t *__restrict__ pos, int64_t ld_pos, int64_t tokens, int Hq, int H,
                int half, int nv, int S, int tok, float sign) {
  extern __shared__ __align__(16) float tab[];  // cos, sin [tok][half]; hi, lo, axis [half]
  pdl_wait();
  pdl_trigger();
  const int64_t t0 = (int64_t)blockIdx.x * tok;
  const int nt = (int)(tokens - t0 < tok ? tokens - t0 : tok);
  float *cs = tab, *sn = tab + tok * half, *hi = sn + tok * half, *lo = hi + half;
  int *axis = reinterpret_cast<int *>(lo + half);
  for (int i = threadIdx.x; i < half; i += kMropeThreads) {
    hi[i] = fr.f.hi[i];
    lo[i] = fr.f.lo[i];
    axis[i] = fr.axis[i];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < nt * half; e += kMropeThreads) {
    const int t = e / half, i = e - t * half;
    const int p = __ldg(pos + (int64_t)axis[i] * ld_pos + t0 + t);
    float c, s;
    rope_cos_sin(p, hi[i], lo[i], &c, &s);
    cs[e] = c;
    sn[e] = sign * s;
  }
  __syncthreads();
  const int w = threadIdx.x / nv, j = threadIdx.x - w * nv, t = w / S, D = 2 * half;
  if (t >= nt) return;
  float c[N], s[N];
  {
    const float *pc = cs + t * half + j * N, *ps = sn + t * half + j * N;
    if constexpr (N % 4 == 0) {
#pragma unroll
      for (int e = 0; e < N; e += 4) {
        *reinterpret_cast<float4 *>(c + e) = *reinterpret_cast<const float4 *>(pc + e);
        *reinterpret_cast<float4 *>(s + e) = *reinterpret_cast<const float4 *>(ps + e);
      }
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        c[e] = pc[e];
        s[e] = ps[e];
      }
    }
  }
  // head h of the Q heads followed by the K heads
  const int64_t row = t0 + t;
  const T *qi = (const T *)q.in + row * q.ld_in + j * N;
  const T *ki = (const T *)k.in + row * k.ld_in + j * N;
  T *qo = (T *)q.out + row * q.ld_out + j * N;
  T *ko = (T *)k.out + row * k.ld_out + j * N;
  for (int h0 = w - t * S; h0 < H; h0 += S * kMropeUnroll<N>) {
    Packet<T, N> a[kMropeUnroll<N>], b[kMropeUnroll<N>];
#pragma unroll
    for (int n = 0; n < kMropeUnroll<N>; ++n) {
      const int h = h0 + n * S;
      if (h < H) {
        const T *src = h < Hq ? qi + (int64_t)h * D : ki + (int64_t)(h - Hq) * D;
        a[n] = load_packet_stream<T, N>(src);
        b[n] = load_packet_stream<T, N>(src + half);
      }
    }
#pragma unroll
    for (int n = 0; n < kMropeUnroll<N>; ++n) {
      const int h = h0 + n * S;
      if (h < H) {
        T *dst = h < Hq ? qo + (int64_t)h * D : ko + (int64_t)(h - Hq) * D;
        turn<T, N>(a[n], b[n], c, s);
        store_packet<T, N>(dst, a[n]);
        store_packet<T, N>(dst + half, b[n]);
      }
    }
  }
}

template <typename T, int N>
cudaError_t launch(const QkMropeArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  MropeFreqs fr;
  fr.f = make_rope_freqs(a.D, a.theta, a.inv_freq);
  const int half = a.D / 2, nv = half / N, H = a.Hq + a.Hkv;
  for (int i = 0; i < kRopeMaxHalf; ++i) fr.axis[i] = i < half ? (uint8_t)a.axis_of[i] : 0;
  // a token's heads go to up to 8 slots of about five heads each (enough heads
  // to pay for a thread's sixteen cosines and sines), the rest of the threads
  // to further tokens; fewer tokens while the grid would not fill the SMs twice
  int S = H / 5 < 1 ? 1 : H / 5 > 8 ? 8 : H / 5;
  int64_t tok = kMropeThreads / (nv * S);
  const int64_t fill = ceil_div(a.T, (int64_t)(2 * dev.sms));
  if (tok > fill) tok = fill;
  if (tok < 1) tok = 1;
  S = kMropeThreads / (nv * (int)tok);
  if (S > H) S = H;
  const int64_t grid = ceil_div(a.T, tok);
  const MropeView q{a.q, a.oq, a.ld_q, a.ld_oq}, k{a.k, a.ok, a.ld_k, a.ld_ok};
  return launch_pdl(qk_mrope_kernel<T, N>, dim3((unsigned)grid), dim3(kMropeThreads),
                    (size_t)(2 * tok + 3) * half * sizeof(float), s, fr, q, k, a.pos, a.ld_pos, a.T, a.Hq,
                    H, half, nv, S, (int)tok, a.backward ? -1.f : 1.f);
}

}  // namespace

cudaError_t launch_qk_mrope(DType dt, bool vec, const QkMropeArgs &a, const DeviceInfo &dev,
                            cudaStream_t s) {
  if (dt == DType::F32) return vec ? launch<float, 4>(a, dev, s) : launch<float, 1>(a, dev, s);
  return vec ? launch<bf16, 8>(a, dev, s) : launch<bf16, 1>(a, dev, s);
}

}  // namespace ftk
