// Dropout of T rows of H features, forward and backward alike:
//   y[t, j] = keep[t, j] ? x[t, j] * scale : 0,   keep from philox.cuh.
// Elementwise: 2 es bytes a column, one generator call for eight.  65,535 x 4,096 bf16:
// 164 us, 6,550 GB/s, 0.98 of the copy rate; 16,384 x 896, which L2 holds, 10.2 us.  fp32:
// 327 us (0.98) and 19.1 (0.92).  The integer work (some 80 instructions for eight columns)
// is hidden behind the memory only because a thread stays with its columns: a part of the
// generator's rounds depends on them alone and is made once (443 us before, by single
// columns and full rounds).
#include "common.cuh"
#include "launch_residual.h"
#include "philox.cuh"
#include "raw_packet.cuh"

namespace ftk {

namespace {

constexpr int kThreads = 256;

// Eight columns: one packet of bf16, two of fp32.
__device__ __forceinline__ void unpack(const uint4 (&u)[1], float2 (&f)[4]) { unpack(u[0], f); }
__device__ __forceinline__ void unpack(const uint4 (&u)[2], float2 (&f)[4]) {
  unpack(u[0], reinterpret_cast<float2(&)[2]>(f[0]));
  unpack(u[1], reinterpret_cast<float2(&)[2]>(f[2]));
}
__device__ __forceinline__ void pack(const float2 (&f)[4], uint4 (&u)[1]) { pack(f, u[0]); }
__device__ __forceinline__ void pack(const float2 (&f)[4], uint4 (&u)[2]) {
  pack(reinterpret_cast<const float2(&)[2]>(f[0]), u[0]);
  pack(reinterpret_cast<const float2(&)[2]>(f[2]), u[1]);
}

// Rows of any alignment: a warp takes 256 columns, each lane making the eight bits of its
// own block, and walks the rows; in a row it walks the columns 32 at a time, so that the
// accesses stay coalesced.  32,767 x 1,001 bf16: 45 us (parts of any row after
// one another 47).
template <typename T>
__global__ void __launch_bounds__(kThreads)
dropout_cols(const T *x, int64_t ldx, T *y, int64_t ldy, int64_t rows, int64_t H, int64_t segs,
             DropArgs d) {
  pdl_wait();
  pdl_trigger();
  const Philox g = philox_of(d);
  const int lane = threadIdx.x & 31;
  // the grid has a warp at least for each of the row's parts
  const int64_t warp = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t step = (int64_t)gridDim.x * (kThreads / 32) / segs;
  const int64_t j0 = warp % segs * 256;
  const PhiloxBlock p = philox_block(g, (uint32_t)(j0 / 8 + lane));
  const uint32_t cut = keep_cut(d.thr);
  for (int64_t t = warp / segs < step ? warp / segs : rows; t < rows; t += step) {
    const T *xr = x + t * ldx + j0 + lane;
    T *yr = y + t * ldy + j0 + lane;
    T v[8];  // all loads first: y may be x, so that the compiler would not move one up
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (j0 + k * 32 + lane < H) v[k] = xr[k * 32];
    uint32_t m = 0xff;
    if (d.thr > 0) m = keep_bits(philox4x32(g, p, philox_row(g, (uint32_t)t)), cut);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t b = __shfl_sync(0xffffffffu, m, k * 4 + lane / 8);
      if (j0 + k * 32 + lane < H)
        yr[k * 32] = from_float<T>(b >> (lane & 7) & 1 ? to_float(v[k]) * d.scale : 0.f);
    }
  }
}

// Rows of whole 16-byte packets: a thread stays with one block of eight columns and
// walks the rows, kRows of them at a time, all loads first.  `cols` threads lie along a
// row (gridDim.y such parts make it up), blockDim.x / cols rows side by side.
constexpr int kRows = kRowsTurn;

template <typename T, bool DROP>
__global__ void __launch_bounds__(kThreads)
dropout_blocks(const T *x, int64_t ldx, T *y, int64_t ldy, int64_t rows, int blocks, int cols,
               DropArgs d) {
  constexpr int kPackets = 8 / VecWidth<T>::value;  // of a block
  pdl_wait();
  pdl_trigger();
  const int r = threadIdx.x / cols, b = blockIdx.y * cols + threadIdx.x - r * cols;
  const int side = blockDim.x / cols;
  if (r >= side || b >= blocks) return;
  const Philox g = philox_of(d);
  const PhiloxBlock p = philox_block(g, (uint32_t)b);
  const uint32_t cut = keep_cut(d.thr);
  const int64_t step = (int64_t)gridDim.x * side;
  for (int64_t t0 = (int64_t)blockIdx.x * side + r; t0 < rows; t0 += kRows * step) {
    uint4 v[kRows][kPackets];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (t0 + i * step < rows)
#pragma unroll
        for (int k = 0; k < kPackets; ++k)
          v[i][k] = load_raw_stream<uint4>(x + (t0 + i * step) * ldx + (int64_t)b * 8 +
                                           k * VecWidth<T>::value);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t t = t0 + i * step;
      if (t < rows) {
        if (DROP) {
          const uint4 u = philox4x32(g, p, philox_row(g, (uint32_t)t));
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
          float2 f[4];
          unpack(v[i], f);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            f[e] = __fmul2_rn(f[e], make_float2(d.scale, d.scale));
            if (!keep_low(w[e], cut)) f[e].x = 0.f;
            if (!keep_high(w[e], cut)) f[e].y = 0.f;
          }
          pack(f, v[i]);
        }
#pragma unroll
        for (int k = 0; k < kPackets; ++k)
          reinterpret_cast<uint4 *>(y + t * ldy + (int64_t)b * 8)[k] = v[i][k];
      }
    }
  }
}

template <typename T>
cudaError_t launch_typed(bool vec, const DropoutArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  if (vec && a.H % 8 == 0) {
    const int blocks = (int)(a.H / 8);
    const int parts = ceil_div(blocks, kThreads), cols = ceil_div(blocks, parts);
    const int side = kThreads / cols;
    const int64_t grid = row_grid(a.T, side, parts, dev);
    auto kern = a.drop.thr > 0 ? dropout_blocks<T, true> : dropout_blocks<T, false>;
    return launch_pdl(kern, dim3((unsigned)grid, (unsigned)parts),
                      dim3((unsigned)(side * cols)), 0, s, (const T *)a.x, a.ldx, (T *)a.y, a.ldy,
                      a.T, blocks, cols, a.drop);
  }
  const int64_t segs = ceil_div(a.H, (int64_t)256);
  int64_t grid = ceil_div(a.T * segs, (int64_t)(kThreads / 32));
  if (grid > (int64_t)dev.sms * 32) grid = (int64_t)dev.sms * 32;
  const int64_t least = ceil_div(segs, (int64_t)(kThreads / 32));
  if (grid < least) grid = least;
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
