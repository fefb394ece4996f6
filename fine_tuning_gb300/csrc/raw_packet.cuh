// Packets of N columns as the residual stream's kernels hold them: the 16 bytes as they
// lie in memory, or one value where columns are single (N = 1), and the same as fp32.
#pragma once

#include "common.cuh"
#include "pair_math.cuh"

namespace ftk {

namespace {

// A packet of N columns as fp32 values: pairs (Blackwell's two-wide fp32 operations,
// each half rounded like the scalar one), or one float where columns are single.
template <int N> struct Values {
  using V = float2;
  static constexpr int kCount = N / 2;
};
template <> struct Values<1> {
  using V = float;
  static constexpr int kCount = 1;
};

__device__ __forceinline__ float vmul(float a, float b) { return a * b; }
__device__ __forceinline__ float2 vmul(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float vfma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float2 vfma(float2 a, float2 b, float2 c) {
  return __ffma2_rn(a, b, c);
}
__device__ __forceinline__ float vsum(float a) { return a; }
__device__ __forceinline__ float vsum(float2 a) { return a.x + a.y; }
template <typename VT> __device__ __forceinline__ VT vall(float a);
template <> __device__ __forceinline__ float vall<float>(float a) { return a; }
template <> __device__ __forceinline__ float2 vall<float2>(float a) { return make_float2(a, a); }

// What a packet is held and moved as: 16 bytes, or one value.
template <typename T, int N> struct Raw {
  using type = uint4;
};
template <typename T> struct Raw<T, 1> {
  using type = T;
};

__device__ __forceinline__ void unpack(const uint4 &u, float2 (&f)[4]) { unpack8(u, f); }
__device__ __forceinline__ void unpack(const uint4 &u, float2 (&f)[2]) {
  f[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
  f[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
}
__device__ __forceinline__ void unpack(float u, float (&f)[1]) { f[0] = u; }
__device__ __forceinline__ void unpack(bf16 u, float (&f)[1]) { f[0] = to_float(u); }
__device__ __forceinline__ void pack(const float2 (&f)[4], uint4 &u) { u = pack8(f); }
__device__ __forceinline__ void pack(const float2 (&f)[2], uint4 &u) {
  u = make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                 __float_as_uint(f[1].y));
}
__device__ __forceinline__ void pack(const float (&f)[1], float &u) { u = f[0]; }
__device__ __forceinline__ void pack(const float (&f)[1], bf16 &u) { u = from_float<bf16>(f[0]); }

template <typename R, typename T> __device__ __forceinline__ R load_raw(const T *p) {
  return *reinterpret_cast<const R *>(p);
}
// for data read once
template <typename R, typename T> __device__ __forceinline__ R load_raw_stream(const T *p) {
  if constexpr (sizeof(R) == 16) {
    R u;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "l"(p));
    return u;
  } else {
    return *p;
  }
}
template <typename R, typename T> __device__ __forceinline__ void store_raw(T *p, const R &u) {
  *reinterpret_cast<R *>(p) = u;
}

}  // namespace

}  // namespace ftk
