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
#include "raw_packet.cuh"

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

// ------------------------------------------------------------------ row groups

// How the register kernels spread rows: W warps a row, V packets of N columns a
// thread (column (gi + k 32W) N + e of thread gi), R rows a CTA.  W = 0: the row does
// not fit, the kernels for any length take it.
struct BlockPlan {
  int V, W, R;
  int threads() const { return 32 * W * R; }
};

constexpr int kMaxWarps = 20;  // of a row group
constexpr int kMaxGroups = 6;  // of more than one warp, in a CTA

// Barrier 1 + g of row group g.  Each case names its barrier by a constant: one computed
// at run time makes the compiler reserve all 16 for every CTA.
__device__ __forceinline__ void row_barrier(int g, int threads) {
  switch (g) {
    case 0: asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory"); break;
    case 1: asm volatile("bar.sync 2, %0;" ::"r"(threads) : "memory"); break;
    case 2: asm volatile("bar.sync 3, %0;" ::"r"(threads) : "memory"); break;
    case 3: asm volatile("bar.sync 4, %0;" ::"r"(threads) : "memory"); break;
    case 4: asm volatile("bar.sync 5, %0;" ::"r"(threads) : "memory"); break;
    default: asm volatile("bar.sync 6, %0;" ::"r"(threads) : "memory"); break;
  }
}

// Packets of 16 bytes: as few a thread as fit, so that the columns' sums and weights stay
// in registers (backward 65,536 x 5,120: one a thread 716 us, two 1,046).  Single columns:
// four a thread where the row has them, since a warp makes the random numbers of 256
// columns at a time (32,767 x 1,001: backward two 234 us, four 155, eight 151, forward
// four 112, eight 116).  Short rows share a CTA of up to `warps`.
inline BlockPlan plan_block_row(int64_t H, int N, int warps) {
  for (int v = N == 1 && H > 32 ? 4 : 1; v <= (N == 1 ? 8 : 4); v *= 2) {
    const int64_t W = ceil_div(H / N, (int64_t)32 * v);
    if (W > kMaxWarps) continue;
    // rows of one warp need no barrier; of the others up to kMaxGroups groups have one each
    const int R = W == 1 || warps / (int)W < kMaxGroups ? warps / (int)W : kMaxGroups;
    return BlockPlan{v, (int)W, R > 0 ? R : 1};
  }
  return BlockPlan{0, 0, 0};
}

// The row group's sums of n values of each thread, to all of them, in a fixed order.
// The values are dealt out while a warp adds its lanes: each step hands half of the
// values to half of the lanes (n = 2 takes 5 shuffles instead of 10, n = 3 6 instead of
// 15, n = 6 9 instead of 30), so that lanes [i L, (i + 1) L) end with value i.  The warps'
// sums meet in slots ([n][kMaxWarps]), which may be written again once every thread has
// passed the group's next barrier.
template <int n> struct Deal {
  static constexpr int kPow = n <= 1 ? 1 : n <= 2 ? 2 : n <= 4 ? 4 : 8;
  static constexpr int L = 32 / kPow;
};

template <int n>
__device__ __forceinline__ void group_sums(float (&v)[n], float *slots, int W, int wig, int grp) {
  constexpr unsigned kAll = 0xffffffffu;
  constexpr int kPow = Deal<n>::kPow, L = Deal<n>::L;
  const int lane = threadIdx.x & 31;
  float d[kPow];
#pragma unroll
  for (int i = 0; i < kPow; ++i) d[i] = i < n ? v[i] : 0.f;
#pragma unroll
  for (int m = kPow / 2, o = 16; m > 0; m /= 2, o /= 2) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < kPow / 2; ++i)
      if (i < m) {
        const float out = up ? d[i] : d[i + m];
        d[i] = (up ? d[i + m] : d[i]) + __shfl_xor_sync(kAll, out, o);
      }
  }
#pragma unroll
  for (int o = L / 2; o > 0; o /= 2) d[0] += __shfl_xor_sync(kAll, d[0], o);
  if (W > 1) {
    const int i = lane / L, sub = lane % L;
    if (sub == 0 && i < n) slots[i * kMaxWarps + wig] = d[0];
    row_barrier(grp, 32 * W);
    d[0] = 0.f;
#pragma unroll
    for (int k = 0; k < (kMaxWarps + L - 1) / L; ++k)
      if (i < n && sub + k * L < W) d[0] += slots[i * kMaxWarps + sub + k * L];
#pragma unroll
    for (int o = L / 2; o > 0; o /= 2) d[0] += __shfl_xor_sync(kAll, d[0], o);
  }
#pragma unroll
  for (int i = 0; i < n; ++i) v[i] = n == 1 ? d[0] : __shfl_sync(kAll, d[0], i * L);
}

// The random numbers of a thread's packets.  A bf16 packet is one call's eight columns,
// an fp32 packet half of them; single columns (N = 1) get their bit from the lanes that
// make the warp's blocks, 4 for each k.
template <int N, int V> struct Mask {
  PhiloxBlock p[V];
  uint32_t cut;
  using Row = uint32_t[V][N / 2];
  __device__ __forceinline__ void init(const Philox &g, int thr, int gi, int G) {
    cut = keep_cut(thr);
#pragma unroll
    for (int k = 0; k < V; ++k) p[k] = philox_block(g, (uint32_t)((gi + k * G) * N / 8));
  }
  __device__ __forceinline__ void row(const Philox &g, uint32_t t, int gi, int G, Row &m) const {
    const uint64_t r = philox_row(g, t);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const uint4 u = philox4x32(g, p[k], r);
      if constexpr (N == 8) {
        m[k][0] = u.x, m[k][1] = u.y, m[k][2] = u.z, m[k][3] = u.w;
      } else {
        const bool odd = (gi + k * G) & 1;
        m[k][0] = odd ? u.z : u.x, m[k][1] = odd ? u.w : u.y;
      }
    }
  }
  // value i of packet k where it is kept, else 0
  __device__ __forceinline__ float2 keep(const Row &m, int k, int i, float2 a) const {
    return make_float2(keep_low(m[k][i], cut) ? a.x : 0.f, keep_high(m[k][i], cut) ? a.y : 0.f);
  }
};
template <int V> struct Mask<1, V> {
  static_assert(V <= 8, "a warp makes 32 blocks");
  PhiloxBlock p;
  uint32_t cut;
  using Row = uint32_t[V];
  __device__ __forceinline__ void init(const Philox &g, int thr, int gi, int G) {
    const int lane = threadIdx.x & 31;
    cut = keep_cut(thr);
    p = philox_block(g, (uint32_t)((gi - lane + (lane >> 2) * G) / 8 + (lane & 3)));
  }
  __device__ __forceinline__ void row(const Philox &g, uint32_t t, int, int, Row &m) const {
    const int lane = threadIdx.x & 31;
    const uint32_t b = keep_bits(philox4x32(g, p, philox_row(g, t)), cut);
#pragma unroll
    for (int k = 0; k < V; ++k)
      m[k] = __shfl_sync(0xffffffffu, b, k * 4 + (lane >> 3)) >> (lane & 7);
  }
  __device__ __forceinline__ float keep(const Row &m, int k, int, float a) const {
    return m[k] & 1 ? a : 0.f;
  }
};

// w_post gate of the packet at column c, as far as they are there.
template <typename T, int N, typename VT>
__device__ __forceinline__ void column_factors(const BlockNorm<T> &a, int64_t c,
                                               VT (&f)[Values<N>::kCount]) {
  using R = typename Raw<T, N>::type;
#pragma unroll
  for (int i = 0; i < Values<N>::kCount; ++i) f[i] = vall<VT>(1.f);
  if (a.w_post != nullptr) unpack(load_raw<R>(a.w_post + c), f);
  if (a.gate != nullptr) {
    VT g[Values<N>::kCount];
    unpack(load_raw<R>(a.gate + c), g);
#pragma unroll
    for (int i = 0; i < Values<N>::kCount; ++i) f[i] = vmul(f[i], g[i]);
  }
}

// Rows of S tensors, walked in steps of one group's rows.  The addresses are uniform in a
// warp (its lanes add a 32-bit offset), and the steps are products that the host made:
// worked out in the loop, they were a sixth of its instructions.
template <int S> struct Walk {
  int64_t step[S];  // bytes from a row of the group to its next
};
template <int S> struct Rows {
  const char *at[S];
  __device__ __forceinline__ void advance(const Walk<S> &w) {
#pragma unroll
    for (int s = 0; s < S; ++s) at[s] += w.step[s];
  }
};

// The row to fetch next, and where in a row the thread's packets lie: `off` bytes from
// its start, each `gap` bytes behind the one before.  With one packet a thread, threads
// past the row's end take its first packet along (with weights of zero, and without
// storing anything), which spares the branches.
struct Turn {
  uint32_t t, step, rows;  // the next row to fetch, the group's step, the batch's rows
  uint32_t off, gap, on;   // bytes; bit k: the thread has a packet k
};

__device__ __forceinline__ uint4 load_shared(uint32_t p) {
  uint4 u;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "r"(p));  // volatile: stays behind the wait for the copies
  return u;
}

// A thread's packets (V of each of S source tensors, B rows at a time) of the rows ahead.
// Packets of 16 bytes are copied into a ring in shared memory (cp.async: each thread
// reads back what it copied itself, so that the ring needs no barrier): kDepth rows, the
// current ones among them.  Single columns, which are too small for such copies, wait in
// registers, one turn ahead.
template <typename T, int N, int V, int S, int B, int kDepth> struct Ahead {
  static_assert(kDepth >= B, "the current rows have to fit");
  static constexpr uint32_t kRow = S * V * 512;  // bytes of a row's packets of one warp
  uint32_t base, cur[B], to;  // shared addresses: the ring, the current rows, the next to fill
  static constexpr size_t bytes(int threads) {
    return (size_t)threads * kDepth * S * V * sizeof(uint4);
  }
  __device__ __forceinline__ uint32_t after(uint32_t p) const {
    return p == base + (kDepth - 1) * kRow ? base : p + kRow;
  }
  __device__ __forceinline__ void fetch(Rows<S> &src, const Walk<S> &w, Turn &n) {
    if (n.t < n.rows)
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (V == 1 || n.on >> k & 1)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + (s * V + k) * 512),
                         "l"(src.at[s] + (n.off + k * n.gap))
                         : "memory");
    cp_async_commit();  // a group for each row, empty or not
    n.t += n.step;
    src.advance(w);
    to = after(to);
  }
  __device__ __forceinline__ void start(uint4 *ring, Rows<S> &src, const Walk<S> &w, Turn &n) {
    base = smem_addr(ring) + (threadIdx.x >> 5) * (kDepth * kRow) + (threadIdx.x & 31) * 16;
    to = cur[0] = base;
#pragma unroll
    for (int b = 1; b < B; ++b) cur[b] = after(cur[b - 1]);
#pragma unroll
    for (int i = 0; i < kDepth - B; ++i) fetch(src, w, n);
  }
  // the current turn's rows are there, kDepth - B rows behind them on their way
  __device__ __forceinline__ void arrive(Rows<S> &src, const Walk<S> &w, Turn &n) {
#pragma unroll
    for (int b = 0; b < B; ++b) fetch(src, w, n);
    cp_async_wait<kDepth - B>();
  }
  __device__ __forceinline__ uint4 get(int s, int b, int k) const {
    return load_shared(cur[b] + (s * V + k) * 512);
  }
  __device__ __forceinline__ void next() {
    cur[0] = after(cur[B - 1]);
#pragma unroll
    for (int b = 1; b < B; ++b) cur[b] = after(cur[b - 1]);
  }
};

template <typename T, int V, int S, int B, int kDepth> struct Ahead<T, 1, V, S, B, kDepth> {
  T now[S][B][V], then[S][B][V];
  static constexpr size_t bytes(int) { return 0; }
  __device__ __forceinline__ void start(uint4 *, Rows<S> &src, const Walk<S> &w, Turn &n) {
#pragma unroll
    for (int b = 0; b < B; ++b) {
      if (n.t < n.rows)
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int k = 0; k < V; ++k)
            if (V == 1 || n.on >> k & 1)
              then[s][b][k] = *reinterpret_cast<const T *>(src.at[s] + (n.off + k * n.gap));
      n.t += n.step;
      src.advance(w);
    }
  }
  __device__ __forceinline__ void arrive(Rows<S> &src, const Walk<S> &w, Turn &n) {
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int b = 0; b < B; ++b)
#pragma unroll
        for (int k = 0; k < V; ++k) now[s][b][k] = then[s][b][k];
    start(nullptr, src, w, n);
  }
  __device__ __forceinline__ T get(int s, int b, int k) const { return now[s][b][k]; }
  __device__ __forceinline__ void next() {}
};

// Where a thread stands: its row group and its place in it.
struct Place {
  int grp, wig, gi, G;
};
__device__ __forceinline__ Place place_of(int W) {
  // from lane 0, so that the compiler knows it to be the same in the whole warp and
  // keeps the row's addresses in uniform registers
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);
  const int grp = warp / W, wig = warp - grp * W;
  return Place{grp, wig, wig * 32 + (int)(threadIdx.x & 31), W * 32};
}

}  // namespace

}  // namespace ftk
