// Attention forward over packed sequences on the 5th-generation tensor cores
// (tcgen05), bf16, head sizes up to 128.
//
//   s = scale q k^T,  o = sum_j e^(s - m) v / l,  lse = m + log l
//
// with the row maximum m and sum l carried along the keys in fp32, so no score
// leaves the SM.  One persistent CTA per SM works on two tiles of 128 query
// rows at a time, both of one key head, so that a staged K or V tile feeds
// two MMAs and one tile's softmax runs under the other's MMAs.  The pair is
// taken along (row tile, head of the group): with an even group both tiles see
// the same keys.  12 warps (one idle):
//   warp 0      one lane issues the TMA tile loads: Q of the pair, then K and V
//               tiles through a ring of kStages;
//   warp 1      one lane issues the MMAs (S = Q K^T from shared memory; O += P V
//               with P read from tensor memory);
//   warps 2-5   softmax of tile 0, one query row per thread (its 128 scores in
//   warps 6-9   registers: no shuffles), and of tile 1;
//   warp 10     zeroes the rows of a V tile that lie behind its sequence's end
//               before the MMAs may read them.
// Tensor memory: S0 S1 (128 columns each) and O0 O1.  P, in bf16, replaces the
// scores it came from.  While softmax t works on S_t(i), the tensor pipe runs
// P V of the other tile and that tile's next scores.
//
// The maximum is only raised when a row's scores pass it by more than 2^8
// (kRaise): until then the old one stands, which changes nothing in exact
// arithmetic (o and l carry the same factor) and keeps p <= 256; a raise
// rescales O in tensor memory.  Rounding p to bf16 (2^-8 relative at most, per
// term) is the price of the tensor cores' second product.
#include <cudaTypedefs.h>

#include <cmath>

#include "attn_tc.cuh"

namespace ftk {

namespace attn {

cudaError_t make_head_map(CUtensorMap *map, const void *base, int64_t T, int64_t H, int64_t D,
                          int64_t ld) {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  if (!encode) {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                                     cudaEnableDefault, &q);
    if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
    encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)ld * 2};
  const cuuint32_t box[3] = {64, 1, kTile};
  const cuuint32_t elem[3] = {1, 1, 1};
  auto make = [&] {
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides,
                  box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = make();
  if (r != CUDA_SUCCESS) {
    // a thread that has made no CUDA call of its own yet (autograd's worker, say)
    // has no current context, which this driver call needs
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaSetDevice(dev);
    if (e != cudaSuccess) return e;
    r = make();
  }
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace attn

namespace {

using namespace attn;

constexpr int kFwdThreads = 384;
constexpr float kRaise = 8.f;  // powers of two

struct FwdParams {
  CUtensorMap tq, tk, tv;
  AttnArgs a;
  int nslots;  // pair slots per key head
};

// Two query tiles of one key head: heads h[], first rows row0[] (within the
// sequence) and key tiles n[] each (0: no such tile).
struct FwdItem {
  int start, len, hk;
  int h[2], row0[2], n[2];
  __device__ __forceinline__ int tiles() const { return max(n[0], n[1]); }
};

// Pairs of (row tile, head of the group) of one sequence: the slots of
// attn_common.cuh with floor((slot G + 1) / 2) + b in place of the slot.
__device__ __forceinline__ int pair_base(int c, int b, int G) {
  return ((max(c, 0) / kTile + b) * G + 1) / 2 + b;
}

__device__ __forceinline__ FwdItem fwd_item(const AttnArgs &a, int nslots, int item) {
  FwdItem w;
  const int G = a.Hq / a.Hkv;
  w.hk = item % a.Hkv;
  // from the last slot back: in one long causal sequence the longest rows first
  const int slot = nslots - 1 - item / a.Hkv;
  int lo = 1, hi = a.B;
  while (lo <= hi) {
    const int mid = (lo + hi) >> 1;
    if (pair_base(__ldg(a.cu + mid), mid, G) <= slot)
      lo = mid + 1;
    else
      hi = mid - 1;
  }
  const int b = min(lo - 1, a.B - 1);
  const int c0 = min(max(__ldg(a.cu + b), 0), (int)a.T);
  const int c1 = min(max(__ldg(a.cu + b + 1), c0), (int)a.T);
  w.start = c0;
  w.len = c1 - c0;
  const int nt = ceil_div(w.len, kTile);
  const int64_t f0 = 2 * ((int64_t)slot - pair_base(c0, b, G));
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int64_t f = f0 + t;
    const bool in = f0 >= 0 && f < (int64_t)nt * G;
    const int tile = in ? (int)(f / G) : 0;
    w.h[t] = w.hk * G + (in ? (int)(f - (int64_t)tile * G) : 0);
    w.row0[t] = tile * kTile;
    w.n[t] = !in ? 0 : a.causal ? tile + 1 : nt;
  }
  return w;
}

template <int DP> struct FwdLayout {
  static constexpr uint32_t tile_bytes = (DP / 64) * kBoxBytes;
  static constexpr int kStages = DP == 128 ? 5 : 8;
  static constexpr uint32_t off_ring = 2 * tile_bytes;
  static constexpr uint32_t off_bar = off_ring + kStages * tile_bytes;
  static constexpr uint32_t smem = off_bar + (3 * kStages + 13) * 8 + 16 + 1024;
  static_assert(smem <= 227 * 1024, "shared memory per CTA");
};

template <int DP>
__global__ void __launch_bounds__(kFwdThreads, 1)
attn_fwd_tc(const __grid_constant__ FwdParams p, unsigned *status, long long wait_limit) {
  using L = FwdLayout<DP>;
  constexpr int kStages = L::kStages;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *sm = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_addr(sm);
  uint64_t *kv_full = reinterpret_cast<uint64_t *>(sm + L::off_bar);
  uint64_t *kv_empty = kv_full + kStages;
  uint64_t *v_ready = kv_empty + kStages;  // the tail warp has seen the stage
  uint64_t *q_full = v_ready + kStages;    // [2] each from here
  uint64_t *q_empty = q_full + 2;
  uint64_t *s_full = q_empty + 2;
  uint64_t *p_full = s_full + 2;
  uint64_t *o_full = p_full + 2;
  uint64_t *o_empty = o_full + 2;
  uint64_t *drain = o_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 2);  // the MMAs and the tail warp
      mbar_init(&v_ready[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 1);
      mbar_init(&q_empty[t], 1);
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 4);
      mbar_init(&o_full[t], 1);
      mbar_init(&o_empty[t], 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc1(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Waits wait{abort_flag, status, wait_limit};
  const AttnArgs &a = p.a;
  pdl_wait();
  pdl_trigger();
  const int items = attn_skipped(a.skip) ? 0 : p.nslots * a.Hkv;

  if (warp == 0) {
    // -------------------------------------------------------- tile loads
    int it = 0, nq[2] = {0, 0};
    bool ok = true;
    auto load_kv = [&](const CUtensorMap *map, int head, int row) {
      const int s = it % kStages;
      ok = wait.all(&kv_empty[s], ((it / kStages) & 1) ^ 1);
      if (!ok) return;
      if (elect_one())
        load_tile<DP>(sbase + L::off_ring + s * L::tile_bytes, map, head, row, &kv_full[s]);
      __syncwarp();
      ++it;
    };
    for (int w = blockIdx.x; ok && w < items; w += gridDim.x) {
      const FwdItem x = fwd_item(a, p.nslots, w);
      const int n = x.tiles();
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (!ok || x.n[t] == 0) continue;
        ok = wait.all(&q_empty[t], (nq[t] & 1) ^ 1);
        if (!ok) break;
        if (elect_one())
          load_tile<DP>(sbase + t * L::tile_bytes, &p.tq, x.h[t], x.start + x.row0[t], &q_full[t]);
        __syncwarp();
        ++nq[t];
      }
      for (int i = 0; ok && i < n; ++i) {
        load_kv(&p.tk, x.hk, x.start + i * kTile);
        if (ok) load_kv(&p.tv, x.hk, x.start + i * kTile);
      }
    }
    // every load has landed before the CTA may leave
    for (int t = 0; t < 2; ++t)
      if (nq[t]) mbar_wait_bounded(&q_full[t], (nq[t] - 1) & 1, wait_limit, status);
    for (int i = max(it - kStages, 0); i < it; ++i)
      mbar_wait_bounded(&kv_full[i % kStages], (i / kStages) & 1, wait_limit, status);
  } else if (warp == 1) {
    // -------------------------------------------------------- MMAs
    const int nk = (a.D + 15) / 16, no = nk * 16;  // contraction steps of S, columns of O
    int it = 0, nq[2] = {0, 0}, np[2] = {0, 0};
    bool ok = true;
    for (int w = blockIdx.x; ok && w < items; w += gridDim.x) {
      const FwdItem x = fwd_item(a, p.nslots, w);
      const int n = x.tiles();
      if (n == 0) continue;
      // scores of key tile i (in `stage`) against query tile t
      auto scores = [&](int t, int i, int stage) {
        if (elect_one()) {
          mma_rows(tmem + t * 128, sbase + t * L::tile_bytes,
                   sbase + L::off_ring + stage * L::tile_bytes, nk);
          mma_commit(&s_full[t]);
          if (i == x.n[t] - 1) mma_commit(&q_empty[t]);  // the last use of this Q tile
        }
        __syncwarp();
      };
      int sk = it % kStages;
      ok = wait.all(&kv_full[sk], (it / kStages) & 1);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (!ok || x.n[t] == 0) continue;
        ok = wait.all(&q_full[t], nq[t] & 1);
        if (!ok) break;
        tc_fence_after();
        scores(t, 0, sk);
      }
      if (!ok) break;
      if (elect_one()) mma_commit(&kv_empty[sk]);
      __syncwarp();
      ++it;
      for (int i = 0; ok && i < n; ++i) {
        const int sv = it % kStages;  // V of tile i, then K of tile i + 1
        // the load first: it came after kv_empty of the stage's last use, hence
        // after that use's v_ready, so the second wait sees no older phase
        ok = wait.all(&kv_full[sv], (it / kStages) & 1) &&
             wait.all(&v_ready[sv], (it / kStages) & 1);
        if (!ok) break;
        ++it;
        const bool more = i + 1 < n;
        sk = it % kStages;
        if (more) {
          ok = wait.all(&kv_full[sk], (it / kStages) & 1);
          if (!ok) break;
          ++it;
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok || i >= x.n[t]) continue;
          ok = wait.all(&p_full[t], np[t] & 1);
          if (ok && i == 0) ok = wait.all(&o_empty[t], (nq[t] & 1) ^ 1);
          if (!ok) break;
          ++np[t];
          tc_fence_after();
          if (elect_one()) {
            mma_prob(tmem + 256 + t * DP, tmem + t * 128,
                     sbase + L::off_ring + sv * L::tile_bytes, no, i != 0);
            mma_commit(&o_full[t]);
          }
          __syncwarp();
          if (i + 1 < x.n[t]) scores(t, i + 1, sk);
        }
        if (!ok) break;
        if (elect_one()) {
          mma_commit(&kv_empty[sv]);
          if (more) mma_commit(&kv_empty[sk]);
        }
        __syncwarp();
      }
      nq[0] += x.n[0] != 0;
      nq[1] += x.n[1] != 0;
    }
    if (it) {  // every MMA issued has completed
      if (elect_one()) mma_commit(drain);
      __syncwarp();
      mbar_wait_bounded(drain, 0, wait_limit, status);
    }
  } else if (warp == 10) {
    // -------------------------------------------------------- V tiles' tails
    int it = 0;
    bool ok = true;
    for (int w = blockIdx.x; ok && w < items; w += gridDim.x) {
      const FwdItem x = fwd_item(a, p.nslots, w);
      const int n = x.tiles();
      for (int i = 0; i < 2 * n; ++i, ++it) {  // K0 V0 K1 V1 ..., as loaded
        const int s = it % kStages;
        ok = wait.all(&kv_full[s], (it / kStages) & 1);
        if (!ok) break;
        const int valid = x.len - (i >> 1) * kTile;
        if ((i & 1) && valid < kTile)
          zero_rows<DP>(sm + L::off_ring + s * L::tile_bytes, valid, lane);
        if (lane == 0) {
          mbar_arrive(&v_ready[s]);  // before kv_empty: see the MMA warp's wait
          mbar_arrive(&kv_empty[s]);
        }
        __syncwarp();
      }
    }
  } else if (warp < 10) {
    // -------------------------------------------------------- softmax
    const int t = (warp - 2) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t ts = tmem + t * 128 + lanes, to = tmem + 256 + t * DP + lanes;
    const float s2 = a.scale * kLog2E;
    int np = 0;
    bool ok = true;
    for (int w = blockIdx.x; ok && w < items; w += gridDim.x) {
      const FwdItem x = fwd_item(a, p.nslots, w);
      const int n = x.n[t];
      if (n == 0) continue;
      const int row = x.row0[t] + r;                              // within the sequence
      const int last = a.causal ? min(row, x.len - 1) : x.len - 1;  // the last key seen
      const int last_all = a.causal ? min(x.row0[t], x.len - 1) : x.len - 1;  // by every row
      float m = -INFINITY, ms = 0.f;
      float2 l2 = make_float2(0.f, 0.f);
      for (int i = 0; i < n; ++i, ++np) {
        ok = wait.all(&s_full[t], np & 1);
        if (!ok) break;
        tc_fence_after();
        uint32_t s[2][64];
        tmem_ld64(ts, s[0]);
        tmem_ld64(ts + 64, s[1]);
        if (i * kTile + kTile - 1 > last_all) {
          const int lim = last - i * kTile;
#pragma unroll
          for (int c = 0; c < kTile; ++c)
            if (c > lim) s[c >> 6][c & 63] = 0xff800000u;  // -inf
        }
        float mx[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = __uint_as_float(s[0][e]);
#pragma unroll
        for (int c = 4; c < kTile; ++c)
          mx[c & 3] = fmaxf(mx[c & 3], __uint_as_float(s[c >> 6][c & 63]));
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        if (i == 0) {
          m = top;
          ms = m == -INFINITY ? 0.f : m * s2;
        } else if (__any_sync(0xffffffffu, (top - m) * s2 > kRaise)) {
          const float mn = fmaxf(m, top);
          const float ns = mn == -INFINITY ? 0.f : mn * s2;
          const float f = ex2(m * s2 - ns);
          ok = wait.all(&o_full[t], (np - 1) & 1);  // P V of the tile before is in O
          if (!ok) break;
          tc_fence_after();
          __syncwarp();
#pragma unroll
          for (int c = 0; c < DP; c += 32) {
            uint32_t o[32];
            tmem_ld32(to + c, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(to + c, o);
          }
          l2.x *= f;
          l2.y *= f;
          m = mn;
          ms = ns;
        }
        __syncwarp();
        const float2 sc = make_float2(s2, s2), off = make_float2(-ms, -ms);
#pragma unroll
        for (int c = 0; c < kTile; c += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const int g = c + e;
            float2 v = make_float2(__uint_as_float(s[g >> 6][g & 63]),
                                   __uint_as_float(s[g >> 6][(g & 63) + 1]));
            v = __ffma2_rn(v, sc, off);
            v.x = ex2(v.x);
            v.y = ex2(v.y);
            l2 = __fadd2_rn(l2, v);
            pk[e >> 1] = pack_bf16(v.x, v.y);
          }
          tmem_st16(ts + (c >> 1), pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t]);
      }
      if (!ok) break;
      ok = wait.all(&o_full[t], (np - 1) & 1);
      if (!ok) break;
      tc_fence_after();
      const float l = l2.x + l2.y, inv = 1.f / l;
      const bool in = row < x.len;
      bf16 *o = (bf16 *)a.o + (int64_t)(x.start + row) * a.ld_o + (int64_t)x.h[t] * a.D;
      // the whole row first, the warp converged, then the divergent stores: a
      // tensor-memory load must never sit behind a branch that lanes take apart
      uint32_t v[DP / 64][64];
      __syncwarp();
#pragma unroll
      for (int j = 0; j < DP / 64; ++j) tmem_ld64(to + 64 * j, v[j]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_empty[t]);  // the next pair's O may be written
      if (in) {
#pragma unroll
        for (int c = 0; c < DP; c += 8) {
          if (c < a.D) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(v[c >> 6][(c & 63) + e]) * inv;
            *reinterpret_cast<uint4 *>(o + c) =
                make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                           pack_bf16(f[6], f[7]));
          }
        }
      }
      if (in && a.lse)
        a.lse[(int64_t)x.h[t] * a.T + x.start + row] = ms * kLn2 + logf(l);
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc1(tmem, 512);
  }
}

template <int DP>
cudaError_t launch(const AttnArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  FwdParams p;
  p.a = a;
  const int64_t G = a.Hq / a.Hkv;
  p.nslots = (int)(((a.T / kTile + a.B) * G + 1) / 2 + a.B);
  cudaError_t e = make_head_map(&p.tq, a.q, a.T, a.Hq, a.D, a.ld_q);
  if (e == cudaSuccess) e = make_head_map(&p.tk, a.k, a.T, a.Hkv, a.D, a.ld_k);
  if (e == cudaSuccess) e = make_head_map(&p.tv, a.v, a.T, a.Hkv, a.D, a.ld_v);
  unsigned *status = nullptr;
  if (e == cudaSuccess) e = device_status_ptr(dev, &status);
  if (e != cudaSuccess) return e;
  constexpr size_t smem = FwdLayout<DP>::smem;
  blocks_per_sm((const void *)attn_fwd_tc<DP>, kFwdThreads, smem, dev, 1);  // lifts the limit
  const int64_t items = (int64_t)p.nslots * a.Hkv;
  const unsigned grid = (unsigned)(items < dev.sms ? items : dev.sms);
  return launch_pdl(attn_fwd_tc<DP>, dim3(grid), dim3(kFwdThreads), smem, s, p, status,
                    kWaitLimitCycles);
}

}  // namespace

cudaError_t launch_attn_fwd_tc(const AttnArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  return a.D <= 64 ? launch<64>(a, dev, s) : launch<128>(a, dev, s);
}

}  // namespace ftk
