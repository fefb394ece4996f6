// What the forward and the backward of the joint of a block's output with the
// residual stream share (block_norm_fwd.cu, block_norm_bwd.cu):
//   b = x r1 w_post gate gate_tok,   r1 = 1 / sqrt(mean_j x^2 + eps)
//   h = res_scale res + x_scale dropout(b)   (rounded, stored)
//   y = h r2 w,                      r2 = 1 / sqrt(mean_j h^2 + eps)
// Without w_post the block's output is taken as it is (r1 = w_post = 1).
#pragma once

#include "common.cuh"
#include "launch_residual.h"
#include "philox.cuh"

namespace ftk {

namespace {

// Kernel parameters: the arguments with their element types.
template <typename T> struct BlockNorm {
  const T *x;
  int64_t ldx;
  const T *res;
  int64_t ldr;
  const T *w_post, *gate, *w;
  const float *gate_tok;
  T *h;
  int64_t ldh;
  T *y;
  int64_t ldy;
  float *rstd_post, *rstd;
  int64_t rows;
  int H;
  float inv_h, eps, res_scale, x_scale;
  DropArgs drop;
  const T *dy;
  int64_t lddy;
  const T *dh;
  int64_t lddh;
  T *dx;
  int64_t lddx;
  T *dres;
  int64_t lddr;
  float *dgate_tok, *ws;
};

template <typename T> BlockNorm<T> block_norm_params(const BlockNormArgs &a) {
  return BlockNorm<T>{(const T *)a.x,
                      a.ldx,
                      (const T *)a.res,
                      a.ldr,
                      (const T *)a.w_post,
                      (const T *)a.gate,
                      (const T *)a.w,
                      a.gate_tok,
                      (T *)a.h,
                      a.ldh,
                      (T *)a.y,
                      a.ldy,
                      a.rstd_post,
                      a.rstd,
                      a.T,
                      (int)a.H,
                      (float)(1.0 / (double)a.H),
                      a.eps,
                      a.res_scale,
                      a.x_scale,
                      a.drop,
                      (const T *)a.dy,
                      a.lddy,
                      (const T *)a.dh,
                      a.lddh,
                      (T *)a.dx,
                      a.lddx,
                      (T *)a.dres,
                      a.lddr,
                      a.dgate_tok,
                      a.ws};
}

// w_post[j] gate[j], as far as they are there.
template <typename T>
__device__ __forceinline__ float column_factor(const BlockNorm<T> &a, int j) {
  const float p = a.w_post != nullptr ? to_float(a.w_post[j]) : 1.f;
  return a.gate != nullptr ? p * to_float(a.gate[j]) : p;
}

// The sum of one value of each thread of a CTA of `warps` warps, to all of them; in
// a fixed order.  `red` holds a float for each warp.
__device__ __forceinline__ float cta_sum(float v, float *red, int warps) {
  v = warp_sum(v);
  __syncthreads();  // the values of the call before have been read
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < warps; ++i) s += red[i];
  return s;
}

// Calls f(j, kept) for the columns of a row: a warp takes 256 columns at a time, each
// lane makes the bits of its own block of eight, and the columns are walked 32 at a
// time, so that accesses of any alignment stay coalesced.
template <typename F>
__device__ __forceinline__ void for_columns(const Philox &g, int thr, int64_t t, int H, F f) {
  const int lane = threadIdx.x & 31;
  for (int j0 = (int)(threadIdx.x >> 5) * 256; j0 < H; j0 += (int)blockDim.x * 8) {
    const uint32_t m = thr > 0 ? keep_bits(g, thr, (uint32_t)(j0 / 8 + lane), (uint32_t)t) : ~0u;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t b = __shfl_sync(0xffffffffu, m, k * 4 + lane / 8);
      const int j = j0 + k * 32 + lane;
      if (j < H) f(j, (b >> (lane & 7) & 1) != 0);
    }
  }
}

}  // namespace

}  // namespace ftk
