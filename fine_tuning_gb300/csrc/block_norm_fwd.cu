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

template <typename T>
cudaError_t fwd_typed(bool, const BlockNormArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  int64_t grid = a.T < (int64_t)dev.sms * 8 ? a.T : (int64_t)dev.sms * 8;
  cudaError_t e = launch_pdl(block_norm_fwd_any<T>, dim3((unsigned)grid), dim3(kThreads), 0, s,
                             block_norm_params<T>(a));
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_norm_fwd(DType dt, bool vec, const BlockNormArgs &a,
                                  const DeviceInfo &dev, cudaStream_t s) {
  return dt == DType::F32 ? fwd_typed<float>(vec, a, dev, s) : fwd_typed<bf16>(vec, a, dev, s);
}

}  // namespace ftk
