// Embedding lookup with scaling, x[t] = scale W[ids[t]], and the gradient of its
// table, dW[v] = scale sum_{t: ids[t] = v} dx[t].  Tokens whose id lies outside
// [0, V) give a row of zeros and no gradient.
//
// The gradient sums every row's tokens in their order, without atomics on shared sums,
// so that it is bitwise reproducible:
//   1. embed_sort: the tokens are sorted by id, a stable radix sort of (id, t) by one
//      cluster of eight CTAs in one launch; digit counts meet through the cluster's
//      shared memory.  The other CTAs of the launch meanwhile write zeros to rows that no
//      token names (not when the gradient is added to what is there), as many as the
//      sort leaves time for;
//   2. embed_grad: the sorted list is cut into chunks of equal length, however the ids
//      are spread: a warp walks one chunk's rows of dx for 256 columns and keeps the
//      running sum of one id in registers.  Sums of ids that lie inside the chunk go to
//      dW, those that cross its borders to the workspace.  Warps between them write the
//      other rows' zeros, which is most of the work where the vocabulary is larger than
//      the batch;
//   3. embed_join: the crossing sums are added in the chunks' order.
//
// Bound by memory, over 151,936 ids: lookup of 65,536 x 4,096 bf16 116 us, 0.92 of the copy
// rate with every named row read once; of 32,768 x 4,096 fp32 128 us, 0.88; rows that are
// not whole packets move two bytes at a time (32,767 x 1,001 49 us, 0.28).  Gradient: 16,384
// x 896 98 us, 5,830 GB/s, 0.87; two parts of 32,768 x 5,120, the second accumulated, 726
// us, 0.88; fp32 16,384 x 896 105 us (0.86), 32,768 x 4,096 460 (0.98); bf16 32,767 x 1,001
// 156 (0.65).  The first form (a launch for each step of the sort, one for the zeros, a CTA
// a chunk) took 181 and 1,814 for the first two.  What does not scale: the sort is eight
// CTAs, for which an accumulating call waits (20 us for 32,768 tokens; 524,288 x 896 537 us,
// 0.52), and a run of one id is joined by one warp for 256 columns (131,072 x 896 191 us,
// with 30% of the batch one id 240).  Spills of embed_grad: 4 to 28 bytes a thread.
#include "common.cuh"
#include "launch_residual.h"
#include "raw_packet.cuh"

namespace ftk {

namespace {

constexpr int kThreads = 256;

// A thread stays with one packet of columns and walks the rows, kRows of them at a time:
// all their ids first, then all their packets.  `cols` threads lie along a row
// (gridDim.y such parts make it up), blockDim.x / cols rows side by side.
constexpr int kRows = kRowsTurn;

template <typename T, int N>
__global__ void __launch_bounds__(kThreads)
embed_fwd_rows(const T *w, int64_t ldw, uint32_t V, const int32_t *ids, T *x, int64_t ldx,
               int64_t rows, int hp, int cols, float scale) {
  using VT = typename Values<N>::V;
  using Rw = typename Raw<T, N>::type;
  constexpr int P = Values<N>::kCount;
  pdl_wait();
  pdl_trigger();
  const int r = threadIdx.x / cols, c = blockIdx.y * cols + threadIdx.x - r * cols;
  const int side = blockDim.x / cols;
  if (c >= hp) return;
  w += (int64_t)c * N;
  x += (int64_t)c * N;
  const int64_t step = (int64_t)gridDim.x * side;
  for (int64_t t0 = (int64_t)blockIdx.x * side + r; t0 < rows; t0 += kRows * step) {
    uint32_t id[kRows];
    Rw v[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      id[i] = t0 + i * step < rows ? (uint32_t)ids[t0 + i * step] : V;
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (id[i] < V) v[i] = load_raw<Rw>(w + (int64_t)id[i] * ldw);  // as unsigned: never < 0
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (t0 + i * step < rows) {
        VT f[P];
        if (id[i] < V) {
          unpack(v[i], f);
#pragma unroll
          for (int e = 0; e < P; ++e) f[e] = vmul(f[e], vall<VT>(scale));
        } else {
#pragma unroll
          for (int e = 0; e < P; ++e) f[e] = vall<VT>(0.f);
        }
        pack(f, v[i]);
        store_raw(x + (t0 + i * step) * ldx, v[i]);
      }
  }
}

template <typename T, int N>
cudaError_t fwd_typed(const EmbedFwdArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  const int hp = (int)(a.H / N), parts = ceil_div(hp, kThreads), cols = ceil_div(hp, parts);
  const int side = kThreads / cols;
  const int64_t grid = row_grid(a.T, side, parts, dev);
  cudaError_t e = launch_pdl(embed_fwd_rows<T, N>, dim3((unsigned)grid, (unsigned)parts),
                             dim3((unsigned)(side * cols)), 0, s, (const T *)a.w, a.ldw,
                             (uint32_t)a.V, a.ids, (T *)a.x, a.ldx, a.T, hp, cols, a.scale);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// ------------------------------------------------------------------- the sort

constexpr int kDigitBits = 9;  // at most, of one pass
constexpr int kDigits = 1 << kDigitBits;
constexpr int kSortThreads = 512;  // a thread for each digit
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortCtas = 8;       // of the cluster
constexpr int64_t kZeroBytes = 128 << 20;  // written beside the sort at least
constexpr int64_t kLongSums = 12 << 20;    // elements of dx
constexpr int kFlagWords = 8192;   // of a zeroing CTA: 32 rows each
constexpr int kColumns = 256;      // of a warp of embed_grad

// Everything that follows from the sizes: passes of the sort, chunks of the sums, and
// where their data lie in the workspace.
struct EmbedPlan {
  int passes, digit_bits;
  int64_t chunks, chunk;  // sums: chunks, tokens of each
  size_t off_key[2], off_tok[2], off_part, bytes;
};

EmbedPlan plan_embed(int64_t T, int64_t H, int64_t V) {
  EmbedPlan p;
  int bits = 1;
  while ((V >> bits) != 0) ++bits;  // V itself marks the tokens without a row
  p.passes = (bits + kDigitBits - 1) / kDigitBits;
  p.digit_bits = (bits + p.passes - 1) / p.passes;
  // Some 8,192 warps in all, 54 an SM.  Measured, 131,072 x 4,096: 727 us, with 4,096
  // warps 822; in the present form 646, with 12,288 657.  16 tokens at least, since each
  // border may cost two rows of fp32 sums.
  p.chunk = ceil_div(ceil_div(T * ceil_div(H, (int64_t)kColumns), (int64_t)8192), (int64_t)8) * 8;
  if (p.chunk < 16) p.chunk = 16;
  if (p.chunk > 1024) p.chunk = 1024;
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
  p.off_part = take((size_t)p.chunks * 2 * (size_t)H * 4);
  p.bytes = at;
  return p;
}

struct SortParams {
  const uint32_t *ids;
  uint32_t V;
  uint32_t n;
  int passes, digit_bits;
  uint32_t *key[2], *tok[2];
  // the rows to zero (zero_ctas > 0): those below zero_rows
  int zero_ctas;  // a power of two
  uint32_t zero_rows;
  float *dw;
  int64_t lddw, H;
};

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();  // the aligned forms want whole warps
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A word of the shared memory of the cluster's CTA `cta`, at this CTA's address `p`.
__device__ __forceinline__ uint32_t cluster_load(const uint32_t *p, int cta) {
  uint32_t at, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(cta));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

constexpr int kSortBatch = 4;  // keys of a lane in flight

// The sort.  In each pass every warp counts the digits of its run of the list; digit d of
// CTA c begins after every smaller digit of all CTAs and after digit d of the CTAs before
// c; inside the CTA the warps' runs follow one another, and inside a warp the order is
// kept by ranks among the lanes of equal digit.
__device__ void sort_tokens(const SortParams &a, uint32_t *shared) {
  uint32_t(*at)[kDigits] = reinterpret_cast<uint32_t(*)[kDigits]>(shared);  // [kSortWarps]
  uint32_t *tot = shared + kSortWarps * kDigits;                            // [kDigits]
  uint32_t *warp_total = tot + kDigits;                                     // [kSortWarps]
  const int cta = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t mask = (1u << a.digit_bits) - 1;
  // runs of whole warps' steps, the last ones shorter or empty
  const uint32_t per = ceil_div(ceil_div(a.n, (uint32_t)(kSortCtas * kSortWarps)), 32u) * 32;
  const uint64_t first = (uint64_t)(cta * kSortWarps + warp) * per;
  const uint32_t lo = first < a.n ? (uint32_t)first : a.n, hi = a.n - lo < per ? a.n : lo + per;
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.digit_bits;
    const uint32_t *keys = pass == 0 ? a.ids : a.key[(pass - 1) & 1];
    const uint32_t *toks = a.tok[(pass - 1) & 1];
    uint32_t *out_key = a.key[pass & 1], *out_tok = a.tok[pass & 1];
    // from L2: other CTAs wrote the keys of a later pass.  Out of range as unsigned, a
    // negative id is beyond V too; V itself is behind every id.
    auto load = [&](uint32_t i) { return min(__ldcg(keys + i), a.V); };
    for (int i = threadIdx.x; i < kSortWarps * kDigits; i += kSortThreads) (&at[0][0])[i] = 0;
    __syncthreads();
    for (uint32_t i = lo + lane; i < hi; i += 32 * kSortBatch) {
      uint32_t k[kSortBatch];
#pragma unroll
      for (int b = 0; b < kSortBatch; ++b)
        if (i + 32 * b < hi) k[b] = load(i + 32 * b);
#pragma unroll
      for (int b = 0; b < kSortBatch; ++b)
        if (i + 32 * b < hi) atomicAdd(&at[warp][k[b] >> shift & mask], 1u);
    }
    __syncthreads();
    uint32_t own = 0;  // of this thread's digit
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) own += at[w][threadIdx.x];
    tot[threadIdx.x] = own;
    cluster_sync();
    uint32_t total = 0, before = 0;
#pragma unroll
    for (int c = 0; c < kSortCtas; ++c) {
      const uint32_t v = cluster_load(tot + threadIdx.x, c);
      if (c < cta) before += v;
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
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const uint32_t v = at[w][threadIdx.x];
      at[w][threadIdx.x] = base;
      base += v;
    }
    __syncthreads();
    for (uint32_t i0 = lo; i0 < hi; i0 += 32 * kSortBatch) {  // uniform in the warp
      uint32_t k[kSortBatch], t[kSortBatch];
#pragma unroll
      for (int b = 0; b < kSortBatch; ++b) {
        const uint32_t i = i0 + 32 * b + lane;
        k[b] = i < hi ? load(i) : 0;
        t[b] = i < hi && pass > 0 ? __ldcg(toks + i) : i;
      }
#pragma unroll
      for (int b = 0; b < kSortBatch; ++b) {
        const bool on = i0 + 32 * b + lane < hi;
        // a digit of its own for the lanes past the end
        const uint32_t d = on ? k[b] >> shift & mask : kDigits;
        const uint32_t same = __match_any_sync(0xffffffffu, d);
        const uint32_t rank = __popc(same & ((1u << lane) - 1));
        uint32_t to = 0;
        if (on) to = at[warp][d] + rank;
        __syncwarp();
        if (on && rank == 0) at[warp][d] += __popc(same);
        __syncwarp();
        if (on) {
          out_key[to] = k[b];
          out_tok[to] = t[b];
        }
      }
    }
    cluster_sync();  // the pass is written, and tot has been read by all
  }
}

// A row of zeros, by a warp: 16 bytes a lane from the first aligned column on, whatever
// the row's alignment.
__device__ __forceinline__ void zero_row(float *row, int64_t H, int lane) {
  const int64_t head = min(H, (int64_t)(-(intptr_t)((uintptr_t)row / 4) & 3));
  const int64_t packets = (H - head) / 4, tail = H - head - 4 * packets;
  if (lane < head) row[lane] = 0.f;
  float4 *body = reinterpret_cast<float4 *>(row + head);
  for (int64_t c = lane; c < packets; c += 32) body[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (lane < tail) row[head + 4 * packets + lane] = 0.f;
}

// Zeros in the rows that no token names.  CTA z has the rows whose number / 32 is z modulo
// zero_ctas (present and absent rows gather at different ends of a vocabulary); it marks
// its rows that the batch names, then its warps fill the others.
__device__ void zero_rows(const SortParams &a, uint32_t *flags) {
  const uint32_t z = blockIdx.x - kSortCtas, Z = a.zero_ctas;
  const int log = 31 - __clz(Z);
  const uint32_t words = (uint32_t)(((uint64_t)a.zero_rows + 31) / 32);
  const uint32_t mine = z < words ? (words - z - 1) / Z + 1 : 0;
  if (mine == 0) return;  // no rows: nothing to look the ids through for
  for (uint32_t i = threadIdx.x; i < mine; i += kSortThreads) flags[i] = 0;
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < a.n; i += kSortThreads * 8) {
    uint32_t id[8];
#pragma unroll
    for (int b = 0; b < 8; ++b)
      id[b] = a.n - i > b * kSortThreads ? a.ids[i + b * kSortThreads] : a.V;
#pragma unroll
    for (int b = 0; b < 8; ++b)
      if (id[b] < a.zero_rows && (id[b] >> 5 & (Z - 1)) == z)
        atomicOr(&flags[id[b] >> 5 >> log], 1u << (id[b] & 31));
  }
  __syncthreads();
  const int lane = threadIdx.x & 31;
  for (uint32_t r = threadIdx.x >> 5; r < mine * 32; r += kSortWarps) {
    const uint64_t v = ((uint64_t)(r >> 5) * Z + z) * 32 + (r & 31);
    if (v < a.zero_rows && !(flags[r >> 5] >> (r & 31) & 1))
      zero_row(a.dw + v * a.lddw, a.H, lane);
  }
}

constexpr size_t kSortShared = sizeof(uint32_t) * (kSortWarps * kDigits + kDigits + kSortWarps);
static_assert(kSortShared >= kFlagWords * sizeof(uint32_t), "the flags lie in the sort's memory");
static_assert(kSortShared <= 48 << 10, "what a launch may have without asking");

__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(kSortThreads, 2)
embed_sort(const SortParams a) {
  extern __shared__ uint32_t shared[];
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x < kSortCtas)
    sort_tokens(a, shared);  // the grid's first cluster
  else
    zero_rows(a, shared);
}

// ------------------------------------------------------------------- the sums

template <typename T> struct GradParams {
  const T *dx;
  int64_t lddx;
  const uint32_t *key, *tok;  // sorted
  uint32_t V, n;
  int chunk, slabs;  // slabs of kColumns columns
  uint32_t units;    // chunks x slabs
  int64_t H;
  float scale;
  float *dw;
  int64_t lddw;
  float *part;  // [chunks][2][H]: the sum that the chunk's first id brings, the last's
  // the rows to zero, from zero_from on: zero_units of kZeroRows, by CTAs spread among the
  // others (of `ctas` in all, `sums` work on units of chunks)
  uint32_t zero_from, zero_units, ctas, sums;
};

// N fp32 values of a row of dW or of a partial sum.
__device__ __forceinline__ void load_f32(const float *p, float2 (&v)[4]) {
  unpack(load_raw<uint4>(p), reinterpret_cast<float2(&)[2]>(v[0]));
  unpack(load_raw<uint4>(p + 4), reinterpret_cast<float2(&)[2]>(v[2]));
}
__device__ __forceinline__ void load_f32(const float *p, float2 (&v)[2]) {
  unpack(load_raw<uint4>(p), v);
}
__device__ __forceinline__ void load_f32(const float *p, float (&v)[1]) { v[0] = *p; }

template <int P> __device__ __forceinline__ void store_f32(float *p, const float2 (&v)[P]) {
#pragma unroll
  for (int i = 0; i < P; i += 2)
    *reinterpret_cast<float4 *>(p + 2 * i) = make_float4(v[i].x, v[i].y, v[i + 1].x, v[i + 1].y);
}
__device__ __forceinline__ void store_f32(float *p, const float (&v)[1]) { *p = v[0]; }

// Adds to global memory without an answer.
template <int P> __device__ __forceinline__ void add_f32(float *p, const float2 (&v)[P]) {
#pragma unroll
  for (int i = 0; i < P; i += 2)
    asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p + 2 * i), "f"(v[i].x),
                 "f"(v[i].y), "f"(v[i + 1].x), "f"(v[i + 1].y)
                 : "memory");
}
__device__ __forceinline__ void add_f32(float *p, const float (&v)[1]) { atomicAdd(p, v[0]); }

__device__ __forceinline__ float vadd(float a, float b) { return a + b; }
__device__ __forceinline__ float2 vadd(float2 a, float2 b) { return __fadd2_rn(a, b); }

// A lane's columns: U packets of N, 32 N apart.
template <typename T, int N> struct Slab {
  static constexpr int U = N == 1 ? 8 : kColumns / (32 * N);
  int64_t c;    // the first column
  uint32_t on;  // bit u: packet u lies in the row
  __device__ __forceinline__ Slab(int slab, int64_t H) {
    c = (int64_t)slab * kColumns + (threadIdx.x & 31) * N;
    on = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) on |= c + u * 32 * N < H ? 1u << u : 0u;
  }
};

// dW's row gets scale * acc, with ACC added to what it holds: by a reduction in L2, which
// needs no answer.  Each element gets one such addition in a call, so that no order can
// change the result.  fp32 reductions in global memory flush subnormal operands and results
// to zero, which the header states.  Measured, and with a load, an addition and a store:
// 32,768 x 5,120 186 and 198 us, 131,072 x 4,096 429 and 507.
template <typename T, int N, bool ACC, typename VT>
__device__ __forceinline__ void finish_row(float *row, const Slab<T, N> &s,
                                           const VT (&acc)[Slab<T, N>::U][Values<N>::kCount],
                                           float scale) {
#pragma unroll
  for (int u = 0; u < Slab<T, N>::U; ++u)
    if (s.on >> u & 1) {
      VT o[Values<N>::kCount];
#pragma unroll
      for (int i = 0; i < Values<N>::kCount; ++i) o[i] = vmul(vall<VT>(scale), acc[u][i]);
      if (ACC)
        add_f32(row + s.c + u * 32 * N, o);
      else
        store_f32(row + s.c + u * 32 * N, o);
    }
}

constexpr int kGradWarps = 4;  // of a CTA
constexpr int kGradCtas = 8;   // of an SM (10, with fewer registers: 8% slower)
constexpr int kZeroRows = 4;  // of a zeroing warp

// Zeros in those of a unit's rows that no token names: each of the first lanes looks one
// id up in the sorted list.
template <typename T>
__device__ void zero_unseen(const GradParams<T> &a, uint32_t unit) {
  if (unit >= a.zero_units) return;
  const int lane = threadIdx.x & 31;
  const uint32_t v0 = a.zero_from + unit * kZeroRows, v = v0 + lane;
  const bool mine = lane < kZeroRows && v < a.V;
  uint32_t lo = 0, hi = mine ? a.n : 0;  // the first place whose key is v or beyond
  while (lo < hi) {
    const uint32_t m = lo + (hi - lo) / 2;
    if (a.key[m] < v) lo = m + 1; else hi = m;
  }
  uint32_t todo = __ballot_sync(0xffffffffu, mine && !(lo < a.n && a.key[lo] == v));
  for (; todo != 0; todo &= todo - 1)
    zero_row(a.dw + (int64_t)(v0 + __ffs(todo) - 1) * a.lddw, a.H, lane);
}

constexpr int kGradBatch = 4;  // rows in flight for a warp

template <typename T, int N, bool ACC>
__global__ void __launch_bounds__(32 * kGradWarps, kGradCtas) embed_grad(const GradParams<T> a) {
  using VT = typename Values<N>::V;
  using Rw = typename Raw<T, N>::type;
  constexpr int U = Slab<T, N>::U, B = kGradBatch, P = Values<N>::kCount;
  constexpr unsigned kAll = 0xffffffffu;
  pdl_wait();
  pdl_trigger();
  uint32_t cta = blockIdx.x;
  if constexpr (!ACC) {
    // CTAs 0 .. ctas - 1 hold the `sums` ones at even distances
    const uint32_t before = (uint32_t)((uint64_t)cta * a.sums / a.ctas);
    if ((uint32_t)((uint64_t)(cta + 1) * a.sums / a.ctas) == before) {
      zero_unseen(a, (cta - before) * kGradWarps + (threadIdx.x >> 5));
      return;
    }
    cta = before;
  }
  const uint32_t unit = cta * kGradWarps + (threadIdx.x >> 5);
  if (unit >= a.units) return;
  const uint32_t ch = unit / a.slabs;
  const Slab<T, N> s(unit - ch * a.slabs, a.H);
  const int lane = threadIdx.x & 31;
  const uint32_t lo = ch * a.chunk, hi = a.n - lo < a.chunk ? a.n : lo + a.chunk;
  uint32_t prev = lo > 0 ? a.key[lo - 1] : a.V;  // the key before the current position
  bool came = true;  // the current run began before this chunk (where prev is its key)
  const T *col = a.dx + s.c;
  VT acc[U][P];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int e = 0; e < P; ++e) acc[u][e] = vall<VT>(0.f);
  float *const part = a.part + (int64_t)ch * 2 * a.H;
  bool some = false;  // acc holds a run's terms
  auto flush = [&](uint32_t k, bool leaves) {
    if (came || leaves) {
      float *p = part + (came ? 0 : a.H) + s.c;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (s.on >> u & 1) store_f32(p + u * 32 * N, acc[u]);
    } else {
      finish_row<T, N, ACC>(a.dw + (int64_t)k * a.lddw, s, acc, a.scale);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < P; ++e) acc[u][e] = vall<VT>(0.f);
  };
  for (uint32_t i0 = lo; i0 < hi; i0 += 32) {
    const uint32_t at = i0 + lane;
    const uint32_t key = at < hi ? a.key[at] : a.V;
    const uint32_t tok = at < hi ? a.tok[at] : 0;
    for (int j0 = 0; j0 < 32 && i0 + j0 < hi; j0 += B) {
      Rw v[B][U];
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const uint32_t k = __shfl_sync(kAll, key, j0 + b);
        const T *p = col + (int64_t)__shfl_sync(kAll, tok, j0 + b) * a.lddx;
        if (k < a.V)
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (s.on >> u & 1) v[b][u] = load_raw_stream<Rw>(p + u * 32 * N);
      }
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const uint32_t k = __shfl_sync(kAll, key, j0 + b);
        if (k != prev) {  // a run ends before this position
          if (some) flush(prev, false);
          came = some = false;
        }
        prev = k;
        if (k < a.V) {
          some = true;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            VT f[P];
            unpack(v[b][u], f);
#pragma unroll
            for (int e = 0; e < P; ++e) acc[u][e] = vadd(acc[u][e], f[e]);
          }
        }
      }
    }
  }
  // the last run: positions past the chunk's end had key V, unless the chunk was full
  if (some) flush(prev, hi < a.n && a.key[hi] == prev);
}

// Joins the sums of an id that crosses chunks: the warp of the chunk where its run begins
// adds the chunks' parts in their order.
template <typename T, int N, bool ACC>
__global__ void __launch_bounds__(32 * kGradWarps) embed_join(const GradParams<T> a) {
  using VT = typename Values<N>::V;
  constexpr int U = Slab<T, N>::U, B = N == 8 ? 8 : N == 4 ? 4 : 2, P = Values<N>::kCount;
  pdl_wait();
  pdl_trigger();
  const uint32_t unit = blockIdx.x * kGradWarps + (threadIdx.x >> 5);
  if (unit >= a.units) return;
  const uint32_t ch = unit / a.slabs;
  const uint32_t lo = ch * a.chunk;
  if (a.n - lo <= a.chunk) return;  // the last chunk
  const uint32_t hi = lo + a.chunk, k = a.key[hi];
  if (k >= a.V || a.key[hi - 1] != k) return;                   // nothing leaves this chunk
  if (lo > 0 && a.key[lo - 1] == k && a.key[lo] == k) return;   // it came in from before
  const Slab<T, N> s(unit - ch * a.slabs, a.H);
  // the last chunk that has a part of it: those from here on that begin with k
  const int lane = threadIdx.x & 31;
  uint32_t last = ch;
  for (;;) {
    const uint64_t c0 = ((uint64_t)last + 1 + lane) * a.chunk;
    const uint32_t out = ~__ballot_sync(0xffffffffu, c0 < a.n && a.key[c0 < a.n ? c0 : 0] == k);
    last += out == 0 ? 32 : __ffs(out) - 1;
    if (out != 0) break;
  }
  VT acc[U][P], v[B][U][P];
  const float *p = a.part + s.c;
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (s.on >> u & 1) load_f32(p + ((int64_t)ch * 2 + 1) * a.H + u * 32 * N, acc[u]);
  for (uint32_t c0 = ch + 1; c0 <= last; c0 += B) {
#pragma unroll
    for (int b = 0; b < B; ++b)
      if (c0 + b <= last)
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (s.on >> u & 1)
            load_f32(p + (int64_t)(c0 + b) * 2 * a.H + u * 32 * N, v[b][u]);
#pragma unroll
    for (int b = 0; b < B; ++b)
      if (c0 + b <= last)
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int e = 0; e < P; ++e) acc[u][e] = vadd(acc[u][e], v[b][u][e]);
  }
  finish_row<T, N, ACC>(a.dw + (int64_t)k * a.lddw, s, acc, a.scale);
}

template <typename T, int N, bool ACC>
cudaError_t bwd_typed(const EmbedBwdArgs &a, cudaStream_t s) {
  const EmbedPlan p = plan_embed(a.T, a.H, a.V);
  unsigned char *const ws = (unsigned char *)a.ws;
  SortParams q{};
  q.ids = (const uint32_t *)a.ids;
  q.V = (uint32_t)a.V;
  q.n = (uint32_t)a.T;
  q.passes = a.T > 0 ? p.passes : 0;
  q.digit_bits = p.digit_bits;
  for (int i = 0; i < 2; ++i) {
    q.key[i] = (uint32_t *)(ws + p.off_key[i]);
    q.tok[i] = (uint32_t *)(ws + p.off_tok[i]);
  }
  if (!ACC) {
    // Long sums want the memory for themselves: all of the zeros beside the sort.  Shorter
    // ones wait for latencies more than for memory: beside the sort about what it leaves time
    // for (some 10 us, and 0.2 us for each 1,024 tokens, at 6 TB/s), the rest beside the sums.
    // Measured, all beside the sort and split, over 151,936 ids: 2,048 x 1,024 112 and 102 us,
    // 4,096 x 2,048 204 and 195, 8,192 x 1,024 115 and 109; 12,288 x 1,024 110 and 113 (ids
    // spread evenly 113 and 113), 4,096 x 4,096 364 and 380, 16,384 x 896 99 and 107, 32,768 x
    // 5,120 526 and 556.  They meet at some 12 million elements, whatever the table's size.
    const int64_t some = kZeroBytes + a.T * 1024, row = 4 * a.H;
    const bool all = a.T * a.H >= kLongSums || a.V <= some / row;
    const int64_t rows = all ? a.V : some / row / 32 * 32;
    q.zero_rows = (uint32_t)(a.T == 0 ? a.V : rows);
    // two waves of two CTAs an SM, which even out (16,384 x 896: 256 106 us, 1,024 102)
    q.zero_ctas = 512;
    const int64_t words = ceil_div((int64_t)q.zero_rows, (int64_t)32);
    while ((int64_t)q.zero_ctas * kFlagWords < words) q.zero_ctas *= 2;
    q.dw = a.dw;
    q.lddw = a.lddw;
    q.H = a.H;
  }
  cudaError_t e = launch_pdl(embed_sort, dim3((unsigned)(kSortCtas + q.zero_ctas)),
                             dim3(kSortThreads), kSortShared, s, q);
  if (e != cudaSuccess || a.T == 0) return e != cudaSuccess ? e : cudaGetLastError();
  const int64_t slabs = ceil_div(a.H, (int64_t)kColumns);
  const int last = (p.passes - 1) & 1;
  GradParams<T> g{(const T *)a.dx, a.lddx, q.key[last], q.tok[last], q.V, q.n,
                  (int)p.chunk, (int)slabs, (uint32_t)(p.chunks * slabs), a.H, a.scale,
                  a.dw, a.lddw, (float *)(ws + p.off_part)};
  g.sums = g.ctas = (uint32_t)ceil_div(p.chunks * slabs, (int64_t)kGradWarps);
  if (!ACC) {
    g.zero_from = q.zero_rows;
    g.zero_units = (uint32_t)ceil_div(a.V - (int64_t)q.zero_rows, (int64_t)kZeroRows);
    g.ctas += (uint32_t)ceil_div((int64_t)g.zero_units, (int64_t)kGradWarps);
  }
  e = launch_pdl(embed_grad<T, N, ACC>, dim3(g.ctas), dim3(32 * kGradWarps), 0, s, g);
  if (e != cudaSuccess) return e;
  e = launch_pdl(embed_join<T, N, ACC>, dim3(g.sums), dim3(32 * kGradWarps), 0, s, g);
  return e != cudaSuccess ? e : cudaGetLastError();
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
  if (dt == DType::F32)
    return vec ? fwd_typed<float, 4>(a, dev, s) : fwd_typed<float, 1>(a, dev, s);
  return vec ? fwd_typed<bf16, 8>(a, dev, s) : fwd_typed<bf16, 1>(a, dev, s);
}

cudaError_t launch_embed_bwd(DType dt, bool vec, const EmbedBwdArgs &a, cudaStream_t s) {
  if (dt == DType::F32) return vec ? bwd_acc<float, 4>(a, s) : bwd_acc<float, 1>(a, s);
  return vec ? bwd_acc<bf16, 8>(a, s) : bwd_acc<bf16, 1>(a, s);
}

}  // namespace ftk
