// Embedding lookup with scaling, x[t] = scale W[ids[t]], and the gradient of its
// table, dW[v] = scale sum_{t: ids[t] = v} dx[t].  Tokens whose id lies outside
// [0, V) give a row of zeros and no gradient.
//
// The gradient sums every row's tokens in their order, without atomics, so that it
// is bitwise reproducible:
//   1. the tokens are sorted by id: a stable radix sort of (id, t), two kernels a
//      digit (counts of each CTA's part; scatter to where the counts say);
//   2. the sorted list is cut into chunks of equal length, however the ids are
//      spread: a CTA walks one chunk's rows of dx for a slab of columns and keeps the
//      running sum of one id in registers.  Sums of ids that lie inside the chunk go
//      to dW, those that cross its borders to the workspace;
//   3. the crossing sums are added in the chunks' order.
// Rows of dW that no token names are set to zero by a kernel of their own (not when
// the gradient is added to what is there).
#include "common.cuh"
#include "launch_residual.h"

namespace ftk {

namespace {

constexpr int kThreads = 256;

template <typename T, int N>
__global__ void __launch_bounds__(kThreads)
embed_fwd_rows(const T *w, int64_t ldw, int64_t V, const int32_t *ids, T *x, int64_t ldx,
               int64_t rows, int hp, float scale) {
  pdl_wait();
  pdl_trigger();
  const int64_t n = rows * hp, step = (int64_t)gridDim.x * kThreads;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += step) {
    const int64_t t = i / hp, c = (i - t * hp) * N;
    const int64_t id = ids[t];
    Packet<T, N> o;
    if (id >= 0 && id < V) {
      const Packet<T, N> v = load_packet<T, N>(w + id * ldw + c);
#pragma unroll
      for (int e = 0; e < N; ++e) o.set(e, v.get(e) * scale);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) o.set(e, 0.f);
    }
    store_packet<T, N>(x + t * ldx + c, o);
  }
}

template <typename T, int N>
cudaError_t fwd_typed(const EmbedFwdArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  const int64_t hp = a.H / N;
  int64_t grid = ceil_div(a.T * hp, (int64_t)kThreads);
  if (grid > (int64_t)dev.sms * 32) grid = (int64_t)dev.sms * 32;
  cudaError_t e = launch_pdl(embed_fwd_rows<T, N>, dim3((unsigned)grid), dim3(kThreads), 0, s,
                             (const T *)a.w, a.ldw, a.V, a.ids, (T *)a.x, a.ldx, a.T, (int)hp,
                             a.scale);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// ------------------------------------------------------------------- the sort

constexpr int kDigitBits = 9;            // at most, of one pass
constexpr int kDigits = 1 << kDigitBits;
constexpr int kSortThreads = 512;        // a thread for each digit
constexpr int kSortWarps = kSortThreads / 32;
constexpr int64_t kSortMaxCtas = 128;
constexpr int64_t kSortMinPart = 2048;   // tokens a CTA sorts at least

// Everything that follows from the sizes: parts of the sort, chunks of the sums, and
// where their data lie in the workspace.
struct EmbedPlan {
  int passes, digit_bits;
  int64_t ctas, part;            // sort: CTAs, tokens of each
  int64_t chunks, chunk;         // sums: chunks, tokens of each
  size_t off_key[2], off_tok[2], off_counts, off_part, bytes;
};

EmbedPlan plan_embed(int64_t T, int64_t H, int64_t V) {
  EmbedPlan p;
  int bits = 1;
  while ((V >> bits) != 0) ++bits;  // V itself marks the tokens without a row
  p.passes = (bits + kDigitBits - 1) / kDigitBits;
  p.digit_bits = (bits + p.passes - 1) / p.passes;
  p.part = ceil_div(ceil_div(T, kSortMaxCtas), kSortMinPart) * kSortMinPart;
  p.ctas = ceil_div(T, p.part);
  p.chunk = ceil_div(T, (int64_t)2048);
  if (p.chunk < 16) p.chunk = 16;
  if (p.chunk > 4096) p.chunk = 4096;  // its keys and tokens stay in shared memory
  p.chunks = ceil_div(T, p.chunk);
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += (n + 255) / 256 * 256;
    return o;
  };
  for (int i = 0; i < 2; ++i) {
    p.off_key[i] = take((size_t)T * 4);
    p.off_tok[i] = take((size_t)T * 4);
  }
  p.off_counts = take((size_t)p.ctas * kDigits * 4);
  p.off_part = take((size_t)p.chunks * 2 * (size_t)H * 4);
  p.bytes = at;
  return p;
}

// The key a token is sorted by: its id, or V (behind every id) where it has no row.
__device__ __forceinline__ uint32_t sort_key(const uint32_t *keys, int64_t i, bool ids,
                                             uint32_t V) {
  const uint32_t k = keys[i];
  return ids && k >= V ? V : k;  // as unsigned, a negative id is beyond V too
}

// counts[cta][digit] of the CTA's part.
__global__ void __launch_bounds__(kSortThreads)
sort_count(const uint32_t *keys, bool ids, uint32_t V, int64_t n, int64_t part, int shift,
           uint32_t mask, uint32_t *counts) {
  __shared__ uint32_t cnt[kDigits];
  for (int d = threadIdx.x; d < kDigits; d += kSortThreads) cnt[d] = 0;
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  const int64_t lo = blockIdx.x * part, hi = lo + part < n ? lo + part : n;
  for (int64_t i = lo + threadIdx.x; i < hi; i += kSortThreads)
    atomicAdd(&cnt[sort_key(keys, i, ids, V) >> shift & mask], 1u);
  __syncthreads();
  for (int d = threadIdx.x; d < kDigits; d += kSortThreads)
    counts[(int64_t)blockIdx.x * kDigits + d] = cnt[d];
}

// Moves the CTA's part to its places: digit d of CTA c begins after every smaller
// digit of all CTAs and after digit d of the CTAs before c; inside the part the
// warps' runs follow one another, and inside a warp the order is kept by ranks
// among the lanes of equal digit.
__global__ void __launch_bounds__(kSortThreads)
sort_scatter(const uint32_t *keys, const uint32_t *toks, bool ids, uint32_t V, int64_t n,
             int64_t part, int shift, uint32_t mask, const uint32_t *counts, uint32_t *out_keys,
             uint32_t *out_toks) {
  __shared__ uint32_t at[kSortWarps][kDigits];
  __shared__ uint32_t warp_total[kSortWarps];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kSortWarps * kDigits; i += kSortThreads) (&at[0][0])[i] = 0;
  // this thread's digit: how many there are, and how many before this CTA's part
  uint32_t total = 0, before = 0;
  for (unsigned c = 0; c < gridDim.x; ++c) {
    const uint32_t v = __ldcg(counts + (int64_t)c * kDigits + threadIdx.x);
    if (c < blockIdx.x) before += v;
    total += v;
  }
  uint32_t incl = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_total[warp] = incl;
  __syncthreads();
  uint32_t base = incl - total + before;
  for (int w = 0; w < warp; ++w) base += warp_total[w];

  const int64_t lo = blockIdx.x * part, hi = lo + part < n ? lo + part : n;
  const int64_t per = ceil_div(hi - lo, (int64_t)kSortThreads) * 32;  // of one warp
  const int64_t wlo = lo + warp * per, whi = wlo + per < hi ? wlo + per : hi;
  for (int64_t i = wlo + lane; i < whi; i += 32)
    atomicAdd(&at[warp][sort_key(keys, i, ids, V) >> shift & mask], 1u);
  __syncthreads();
  for (int w = 0; w < kSortWarps; ++w) {
    const uint32_t v = at[w][threadIdx.x];
    at[w][threadIdx.x] = base;
    base += v;
  }
  __syncthreads();
  for (int64_t i = wlo; i < whi; i += 32) {  // uniform in the warp
    const bool on = i + lane < whi;
    uint32_t k = 0, d = kDigits;  // a digit of its own for the lanes past the end
    if (on) {
      k = sort_key(keys, i + lane, ids, V);
      d = k >> shift & mask;
    }
    const uint32_t same = __match_any_sync(0xffffffffu, d);
    const uint32_t rank = __popc(same & ((1u << lane) - 1));
    uint32_t to = 0;
    if (on) to = at[warp][d] + rank;
    __syncwarp();
    if (on && rank == 0) at[warp][d] += __popc(same);
    __syncwarp();
    if (on) {
      out_keys[to] = k;
      out_toks[to] = toks != nullptr ? toks[i + lane] : (uint32_t)(i + lane);
    }
  }
}

// ------------------------------------------------------------------- the sums

template <typename T, int N> struct GradParams {
  const T *dx;
  int64_t lddx;
  const uint32_t *key, *tok;  // sorted
  uint32_t V;
  int64_t T_, chunk;
  int hp;      // packets of a row
  int64_t H;
  float scale;
  float *dw;
  int64_t lddw;
  float *part;  // [chunks][2][H]: the sum that the chunk's first id brings, the last's
};

template <int N> __device__ __forceinline__ void load_f32(const float *p, float (&v)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int e = 0; e < N; e += 4) {
      const float4 f = *reinterpret_cast<const float4 *>(p + e);
      v[e] = f.x, v[e + 1] = f.y, v[e + 2] = f.z, v[e + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = p[e];
  }
}
template <int N> __device__ __forceinline__ void store_f32(float *p, const float (&v)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int e = 0; e < N; e += 4)
      *reinterpret_cast<float4 *>(p + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) p[e] = v[e];
  }
}

// dW's row gets scale * acc, added to what it holds with ACC.
template <int N, bool ACC>
__device__ __forceinline__ void finish_row(float *p, const float (&acc)[N], float scale) {
  float o[N];
  if (ACC) {
    load_f32<N>(p, o);
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = fmaf(scale, acc[e], o[e]);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = scale * acc[e];
  }
  store_f32<N>(p, o);
}

constexpr int kGradBatch = 8;  // rows of dx in flight for each thread

template <typename T, int N, bool ACC>
__global__ void __launch_bounds__(kThreads) embed_grad(const GradParams<T, N> a) {
  extern __shared__ uint32_t list[];  // [chunk] keys, [chunk] tokens
  pdl_wait();
  pdl_trigger();
  const int64_t lo = blockIdx.x * a.chunk;
  const int n = (int)(lo + a.chunk < a.T_ ? a.chunk : a.T_ - lo);
  uint32_t *key = list, *tok = list + a.chunk;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    key[i] = a.key[lo + i];
    tok[i] = a.tok[lo + i];
  }
  const uint32_t prev = lo > 0 ? a.key[lo - 1] : a.V;
  const uint32_t next = lo + n < a.T_ ? a.key[lo + n] : a.V;
  __syncthreads();
  const int c = blockIdx.y * kThreads + threadIdx.x;
  if (c >= a.hp) return;
  const T *col = a.dx + (int64_t)c * N;
  float acc[N];
#pragma unroll
  for (int e = 0; e < N; ++e) acc[e] = 0.f;
  bool first = prev == key[0];  // the run came in from the chunk before
  for (int i0 = 0; i0 < n; i0 += kGradBatch) {
    Packet<T, N> v[kGradBatch];
#pragma unroll
    for (int b = 0; b < kGradBatch; ++b)
      if (i0 + b < n && key[i0 + b] < a.V)
        v[b] = load_packet_stream<T, N>(col + (int64_t)tok[i0 + b] * a.lddx);
#pragma unroll
    for (int b = 0; b < kGradBatch; ++b) {
      const int i = i0 + b;
      if (i >= n) break;
      const uint32_t k = key[i];
      if (k >= a.V) return;  // only tokens without a row follow
#pragma unroll
      for (int e = 0; e < N; ++e) acc[e] += v[b].get(e);
      const bool last = i + 1 == n;
      if (!last && key[i + 1] == k) continue;
      if (first || (last && next == k)) {
        store_f32<N>(a.part + ((int64_t)blockIdx.x * 2 + (first ? 0 : 1)) * a.H + (int64_t)c * N,
                     acc);
      } else {
        finish_row<N, ACC>(a.dw + (int64_t)k * a.lddw + (int64_t)c * N, acc, a.scale);
      }
      first = false;
#pragma unroll
      for (int e = 0; e < N; ++e) acc[e] = 0.f;
    }
  }
}

// Joins the sums of an id that crosses chunks: the CTA of the chunk where its run
// begins adds the chunks' parts in their order.
template <int N, bool ACC>
__global__ void __launch_bounds__(kThreads)
embed_join(const uint32_t *key, uint32_t V, int64_t n, int64_t chunk, int hp, int64_t H,
           float scale, const float *part, float *dw, int64_t lddw) {
  pdl_wait();
  pdl_trigger();
  const int64_t lo = blockIdx.x * chunk, hi = lo + chunk;  // hi is in the next chunk
  if (hi >= n) return;
  const uint32_t k = key[hi - 1];
  if (k >= V || key[hi] != k) return;                        // nothing leaves this chunk
  if (lo > 0 && key[lo - 1] == k && key[lo] == k) return;    // it came in from before
  const int c = blockIdx.y * kThreads + threadIdx.x;
  if (c >= hp) return;
  float acc[N], v[N];
  load_f32<N>(part + ((int64_t)blockIdx.x * 2 + 1) * H + (int64_t)c * N, acc);
  for (int64_t b = blockIdx.x + 1;; ++b) {
    load_f32<N>(part + b * 2 * H + (int64_t)c * N, v);
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] += v[e];
    const int64_t end = (b + 1) * chunk;
    if (end >= n || key[end] != k) break;
  }
  finish_row<N, ACC>(dw + (int64_t)k * lddw + (int64_t)c * N, acc, scale);
}

// Zeros in the rows that no token names.  Each lane looks one id up in the sorted
// list; the warp then fills its absent rows.
template <int N>
__global__ void __launch_bounds__(kThreads)
embed_zero(const uint32_t *key, int64_t n, int64_t V, int hp, float *dw, int64_t lddw) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t v0 = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * 32;
  if (v0 >= V) return;
  const int64_t v = v0 + lane;
  int64_t lo = 0, hi = n;  // the first place whose key is v or beyond
  while (lo < hi) {
    const int64_t m = (lo + hi) / 2;
    if ((int64_t)key[m] < v) lo = m + 1; else hi = m;
  }
  uint32_t todo = __ballot_sync(0xffffffffu, v < V && !(lo < n && (int64_t)key[lo] == v));
  const float zero[N] = {};
  while (todo != 0) {
    float *row = dw + (v0 + __ffs(todo) - 1) * lddw;
    todo &= todo - 1;
    for (int c = lane; c < hp; c += 32) store_f32<N>(row + (int64_t)c * N, zero);
  }
}

template <typename T, int N, bool ACC>
cudaError_t bwd_typed(const EmbedBwdArgs &a, cudaStream_t s) {
  cudaError_t e;
  const EmbedPlan p = plan_embed(a.T, a.H, a.V);
  unsigned char *const ws = (unsigned char *)a.ws;
  const uint32_t V = (uint32_t)a.V;
  const int hp = (int)(a.H / N);
  uint32_t *key = nullptr, *tok = nullptr;
  if (a.T > 0) {
    uint32_t *const counts = (uint32_t *)(ws + p.off_counts);
    const uint32_t *in_key = (const uint32_t *)a.ids, *in_tok = nullptr;
    for (int i = 0; i < p.passes; ++i) {
      key = (uint32_t *)(ws + p.off_key[i & 1]);
      tok = (uint32_t *)(ws + p.off_tok[i & 1]);
      const int shift = i * p.digit_bits;
      const uint32_t mask = (1u << p.digit_bits) - 1;
      e = launch_pdl(sort_count, dim3((unsigned)p.ctas), dim3(kSortThreads), 0, s, in_key, i == 0,
                     V, a.T, p.part, shift, mask, counts);
      if (e != cudaSuccess) return e;
      e = launch_pdl(sort_scatter, dim3((unsigned)p.ctas), dim3(kSortThreads), 0, s, in_key,
                     in_tok, i == 0, V, a.T, p.part, shift, mask, counts, key, tok);
      if (e != cudaSuccess) return e;
      in_key = key;
      in_tok = tok;
    }
    const GradParams<T, N> g{(const T *)a.dx, a.lddx, key, tok, V,   a.T,    p.chunk,
                             hp,              a.H,    a.scale,  a.dw, a.lddw,
                             (float *)(ws + p.off_part)};
    const dim3 grid((unsigned)p.chunks, (unsigned)ceil_div(hp, kThreads));
    e = launch_pdl(embed_grad<T, N, ACC>, grid, dim3(kThreads), (size_t)p.chunk * 8, s, g);
    if (e != cudaSuccess) return e;
    e = launch_pdl(embed_join<N, ACC>, grid, dim3(kThreads), 0, s, key, V, a.T, p.chunk, hp, a.H,
                   a.scale, g.part, a.dw, a.lddw);
    if (e != cudaSuccess) return e;
  }
  if (!ACC) {
    const int64_t warps = ceil_div(a.V, (int64_t)32);
    e = launch_pdl(embed_zero<N>, dim3((unsigned)ceil_div(warps, (int64_t)(kThreads / 32))),
                   dim3(kThreads), 0, s, key, a.T, a.V, hp, a.dw, a.lddw);
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

template <typename T, int N>
cudaError_t bwd_acc(const EmbedBwdArgs &a, cudaStream_t s) {
  return a.accumulate ? bwd_typed<T, N, true>(a, s) : bwd_typed<T, N, false>(a, s);
}

}  // namespace

size_t embed_bwd_workspace_bytes(int64_t T, int64_t H, int64_t V) {
  return T > 0 ? plan_embed(T, H, V).bytes : 256;
}

cudaError_t launch_embed_fwd(DType dt, bool vec, const EmbedFwdArgs &a, const DeviceInfo &dev,
                             cudaStream_t s) {
  if (dt == DType::F32) return vec ? fwd_typed<float, 4>(a, dev, s) : fwd_typed<float, 1>(a, dev, s);
  return vec ? fwd_typed<bf16, 8>(a, dev, s) : fwd_typed<bf16, 1>(a, dev, s);
}

cudaError_t launch_embed_bwd(DType dt, bool vec, const EmbedBwdArgs &a, const DeviceInfo &,
                             cudaStream_t s) {
  if (dt == DType::F32) return vec ? bwd_acc<float, 4>(a, s) : bwd_acc<float, 1>(a, s);
  return vec ? bwd_acc<bf16, 8>(a, s) : bwd_acc<bf16, 1>(a, s);
}

}  // namespace ftk
