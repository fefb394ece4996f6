// Dropout of T rows of H features, forward and backward alike:
//   y[t, j] = keep[t, j] ? x[t, j] * scale : 0,   keep from philox.cuh.
// Elementwise: 2 es bytes an element, one Philox call for eight.
#include "common.cuh"
#include "launch_residual.h"
#include "philox.cuh"

namespace ftk {

namespace {

constexpr int kThreads = 256;

// A warp takes 256 columns of a row: each lane makes the eight bits of its own
// block, then the warp walks the columns 32 at a time, so that accesses of any
// alignment stay coalesced.
template <typename T>
__global__ void __launch_bounds__(kThreads)
dropout_cols(const T *x, int64_t ldx, T *y, int64_t ldy, int64_t rows, int64_t H, int64_t segs,
             DropArgs d) {
  pdl_wait();
  pdl_trigger();
  const Philox g = philox_of(d);
  const int lane = threadIdx.x & 31;
  const int64_t n = rows * segs, step = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < n; i += step) {
    const int64_t t = i / segs, j0 = (i - t * segs) * 256;
    const uint32_t m = keep_bits(g, d.thr, (uint32_t)(j0 / 8 + lane), (uint32_t)t);
    const T *xr = x + t * ldx + j0;
    T *yr = y + t * ldy + j0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t b = __shfl_sync(0xffffffffu, m, k * 4 + lane / 8);
      const int c = k * 32 + lane;
      if (j0 + c < H)
        yr[c] = from_float<T>(b >> (lane & 7) & 1 ? to_float(xr[c]) * d.scale : 0.f);
    }
  }
}

template <typename T>
cudaError_t launch_typed(bool, const DropoutArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  const int64_t segs = ceil_div(a.H, (int64_t)256);
  int64_t grid = ceil_div(a.T * segs, (int64_t)(kThreads / 32));
  if (grid > (int64_t)dev.sms * 32) grid = (int64_t)dev.sms * 32;
  cudaError_t e = launch_pdl(dropout_cols<T>, dim3((unsigned)grid), dim3(kThreads), 0, s,
                             (const T *)a.x, a.ldx, (T *)a.y, a.ldy, a.T, a.H, segs, a.drop);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_dropout(DType dt, bool vec, const DropoutArgs &a, const DeviceInfo &dev,
                           cudaStream_t s) {
  return dt == DType::F32 ? launch_typed<float>(vec, a, dev, s)
                          : launch_typed<bf16>(vec, a, dev, s);
}

}  // namespace ftk
