// Attention backward over packed sequences on the 5th-generation tensor cores
// (tcgen05), bf16, head sizes up to 128.  The probabilities are recomputed:
//
//   p = e^(scale q k^T - lse),  delta = sum_d do o,  dv = p^T do
//   ds = p (do v^T - delta),    dq = scale ds k,     dk = scale ds^T q
//
// Two kernels after a small one for delta, instead of one that would add its
// dq parts into memory: dq is summed over key tiles and dk, dv over query
// tiles (and over the query heads that share a key head), each inside one
// CTA's tensor memory, in a fixed order, without atomics and without fp32
// partials in HBM.  The price is two more products per tile pair (seven
// instead of five: s and do v^T are made twice); in return the gradients are
// bitwise reproducible and nothing but them is written.
//
// Both kernels have 12 warps: warp 0 issues the tile loads, warp 1 the MMAs,
// warps 2-9 turn scores into probabilities and score gradients (thread = tile
// row, two groups of four warps take a half of the columns each), warp 10
// prepares tails, warp 11 finds the work items.  p and ds go back to tensor
// memory in bf16, over the fp32 values they came from (each half within its own
// 64 columns, so the halves need no barrier between them), and enter the next
// product from there.  The MMAs are queued so that the tensor pipe always has
// the next tile's scores to work on while p and ds are formed: with heads of
// 128 both kernels are bound by the MMAs of their tile pairs (dq: 3, dk/dv: 4,
// 512 cycles each for 128 x 128 x 128; the pipe is busy 69 and 79% of the time),
// with heads of 64 by the exponentials and conversions of the 8 warps (44 and
// 47%).  Measured, one causal sequence of 8,192 tokens, 32/8 heads: 517 us (dq)
// and 637 (dk, dv) with heads of 128, 397 and 523 with heads of 64; 16,384 tokens,
// 32/8 x 128, everything: 4.8 ms.  16 warps on the scores instead of 8: 4% slower;
// the two halves of a tile on barriers and 64-column products of their own, so
// that one half's exponentials run under the other's gradients: 25% slower (64).
#include <cmath>

#include "attn_tc.cuh"

namespace ftk {

namespace {

using namespace attn;

constexpr int kBwdThreads = 384;
constexpr int kComputeWarps = 8;

struct BwdParams {
  CUtensorMap tq, tk, tv, tg, tdq;  // tg: do; tdq: boxes of 32 columns to store
  AttnArgs a;
  int slots;
  int splits;  // CTAs that share a key tile's query heads (dk, dv)
  float *part;  // splits > 1: [splits][dk, dv][T][Hkv][D] sums, unscaled
};

// How many CTAs share the query heads of a key tile.  dk and dv of a key head
// are summed over its group's heads, so a call has T / 128 x Hkv of these sums,
// and the one of a long sequence's first tile passes over all its queries, G
// times: 304 / sums as long as an SM's part of the work (152 SMs, half of the
// tiles masked) if the batch is one sequence.  So many CTAs are given its heads,
// and their fp32 sums (8 bytes per element and share in the workspace) are added
// in order by a small kernel.  Fractions round up by G / 8: the more heads, the
// longer the sum against the fixed cost of a share; by two whole shares at most,
// so that the workspace does not grow with the group.  152 and not the device's
// count: the workspace and the order of the sums follow from the call alone.
// Measured, one CTA per sum against this rule, us: one sequence of 8,192, 8/1 x
// 128: 801, 336; of 2,048, 32/8 x 128: 149, 125 (141 always rounded up); 16,384
// tokens in 85 sequences, 14/2 x 64: 174, 165; 4,096 in 4, 32/8 x 128: 296, 296
// (313 rounded up).  G / 8 without the bound, one share at most, this rule, 38,784
// tokens 64/1: sequences of 4,000 x 128 6,281, 6,580, 6,290; of 200 x 128 1,540,
// 1,434, 1,430; one x 64 37,400, 37,530, 37,660 (9, 2 and 3 shares).
int attn_bwd_splits(int64_t T, int32_t Hq, int32_t Hkv) {
  const int64_t G = Hq / Hkv, sums = ceil_div(T, (int64_t)kTile) * Hkv, want = 2 * 152;
  if (sums >= want) return 1;
  const int64_t n = (8 * want + sums * (G < 16 ? G : 16)) / (8 * sums);
  return (int)(n < G ? n : G);
}

size_t delta_bytes(int64_t T, int32_t Hq) {
  return ((size_t)T * Hq * sizeof(float) + 15) / 16 * 16;
}
float *attn_bwd_part(const AttnArgs &a) {
  return reinterpret_cast<float *>(reinterpret_cast<char *>(a.delta) + delta_bytes(a.T, a.Hq));
}

// acc [128 x n] (+)= P B with P's bf16 halves in columns 0..31 and 64..95 of p.
__device__ __forceinline__ void mma_halves(uint32_t acc, uint32_t p, uint32_t b, int n,
                                           bool accumulate) {
  const uint32_t id = idesc_of(n, true);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    mma_ts(acc, p + (uint32_t)((kk & 3) * 8 + (kk >> 2) * 64), desc_mn(b, kk), id,
           accumulate || kk != 0);
}

// 64 columns of a row, rounded to bf16, to global memory (columns below n).
__device__ __forceinline__ void store_half(bf16 *o, const uint32_t (&v)[64], float f, int n) {
#pragma unroll
  for (int c = 0; c < 64; c += 8) {
    if (c < n) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(v[c + e]) * f;
      *reinterpret_cast<uint4 *>(o + c) =
          make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                     pack_bf16(x[6], x[7]));
    }
  }
}

// Tile of unit u of the whole batch (a SeqTile with len 0: none).  By length
// where that order was made, else in the order of the slots; back: from a sequence's
// last tile on instead of its first.
__device__ __forceinline__ SeqTile tile_of(const AttnArgs &a, int slots, int u, bool back,
                                           const SeqOrder &seqs, bool by_length) {
  if (!by_length) return seq_tile(back ? slots - 1 - u : u, a.cu, a.B, (int)a.T, kTile);
  if (u >= seqs.total) return SeqTile{0, 0, 0};
  const int r = seqs.rank_of(u, a.B), b = seqs.order[r], i = u - seqs.base[r];
  const int c0 = min(max(__ldg(a.cu + b), 0), (int)a.T);
  const int len = min(max(__ldg(a.cu + b + 1), c0), (int)a.T) - c0;
  const int tile = back ? ceil_div(len, kTile) - 1 - i : i;
  return SeqTile{c0, tile >= 0 && tile * kTile < len ? len : 0, tile * kTile};
}

// ------------------------------------------------------------------- delta

// delta[h, t] = sum_d do[t, h, d] o[t, h, d]: L lanes per row, one 16-byte packet
// each, four rows per lane with all loads before the first sum; a warp walks
// consecutive tokens of one head, so delta is written in runs.  Bound by HBM (do
// and o read once): 23 us for 134 MB, 12 for 59 (heads of 64).
template <int L>
__global__ void __launch_bounds__(256) attn_delta_packed(const AttnArgs a) {
  constexpr int kRows = 256 / L;
  pdl_wait();
  pdl_trigger();
  if (attn_skipped(a.skip)) return;
  const int h = blockIdx.x % a.Hq;
  const int64_t t0 = (int64_t)(blockIdx.x / a.Hq) * (4 * kRows) + threadIdx.x / L;
  const int c = threadIdx.x % L * 8;
  const bool in = c < a.D;
  uint4 g[4], o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = t0 + kRows * i;
    g[i] = o[i] = make_uint4(0u, 0u, 0u, 0u);
    if (in && t < a.T) {
      g[i] = *reinterpret_cast<const uint4 *>((const bf16 *)a.do_ + t * a.ld_do +
                                              (int64_t)h * a.D + c);
      o[i] = *reinterpret_cast<const uint4 *>((const bf16 *)a.o + t * a.ld_o + (int64_t)h * a.D + c);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
    const uint32_t y[4] = {o[i].x, o[i].y, o[i].z, o[i].w};
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s = fmaf(__uint_as_float(x[e] << 16), __uint_as_float(y[e] << 16), s);
      s = fmaf(__uint_as_float(x[e] & 0xffff0000u), __uint_as_float(y[e] & 0xffff0000u), s);
    }
#pragma unroll
    for (int w = L / 2; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    const int64_t t = t0 + kRows * i;
    if (threadIdx.x % L == 0 && t < a.T) a.delta[(int64_t)h * a.T + t] = s;
  }
}

// ---------------------------------------------------------------------- dq

// One CTA: 128 query rows of one head against the key tiles they see.
// Tensor memory: S in two buffers, do v^T, dq.  Queue per key tile i, after
// ds(i) is ready: do v^T (i+1), dq += ds(i) K, S(i+2) over ds(i).
template <int DP> struct DqLayout {
  static constexpr uint32_t tile_bytes = (DP / 64) * kBoxBytes;
  static constexpr int kK = DP == 128 ? 3 : 5, kV = DP == 128 ? 2 : 4;
  static constexpr uint32_t off_g = tile_bytes, off_k = 2 * tile_bytes;
  static constexpr uint32_t off_v = off_k + kK * tile_bytes;
  // 2 KB per compute warp; with heads of 128 nothing is left for it
  static constexpr uint32_t off_stage = off_v + kV * tile_bytes;
  static constexpr uint32_t off_bar = off_stage + (DP == 64 ? kComputeWarps * 2048 : 0);
  static constexpr uint32_t off_items = (off_bar + (3 * kK + 2 * kV + 11) * 8 + 16 + 15) / 16 * 16;
  static constexpr uint32_t off_order = off_items + ItemRing::kBytes;
  static constexpr uint32_t smem = off_order + SeqOrder::kBytes + 1024;
  static_assert(smem <= 227 * 1024, "shared memory per CTA");
};

template <int DP>
__global__ void __launch_bounds__(kBwdThreads, 1)
attn_dq_tc(const __grid_constant__ BwdParams p, unsigned *status, long long wait_limit) {
  using L = DqLayout<DP>;
  constexpr int kK = L::kK, kV = L::kV;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *sm = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_addr(sm);
  uint64_t *k_full = reinterpret_cast<uint64_t *>(sm + L::off_bar);
  uint64_t *k_empty = k_full + kK, *k_ready = k_empty + kK;
  uint64_t *v_full = k_ready + kK, *v_empty = v_full + kV;
  uint64_t *q_full = v_empty + kV, *q_empty = q_full + 1;
  uint64_t *s_full = q_empty + 1;  // [2]
  uint64_t *ds_ready = s_full + 2;  // [2]
  uint64_t *dp_full = ds_ready + 2, *acc_full = dp_full + 1, *acc_empty = acc_full + 1;
  uint64_t *drain = acc_empty + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 2);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const ItemRing ring(sm + L::off_items);
  const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kK; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 2);  // the MMAs and the tail warp
      mbar_init(&k_ready[s], 1);
    }
    for (int s = 0; s < kV; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&ds_ready[s], kComputeWarps);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(dp_full, 1);
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, kComputeWarps);
    mbar_init(drain, 1);
    ring.init(11);  // MMAs, eight compute warps, tails
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc1(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  const uint32_t t_dp = tmem + 256, t_dq = tmem + 384;
  const Waits wait{abort_flag, status, wait_limit};
  const AttnArgs &a = p.a;
  pdl_wait();
  pdl_trigger();
  const int G = a.Hq / a.Hkv;
  const bool skipped = attn_skipped(a.skip);
  SeqOrder seqs(sm + L::off_order);
  const bool by_length = a.B > 1 && a.B <= kSortMax;
  if (by_length && !skipped)
    seqs.make(a, reinterpret_cast<int *>(sm), [](int len) { return ceil_div(len, kTile); });
  // index w: head w % Hq (the heads of a group follow each other and share K and
  // V in L2), tiles from the last one back, whose rows see most keys
  auto find = [&](int w, int (&v)[kItemWords]) {
    const SeqTile x = tile_of(a, p.slots, w / a.Hq, true, seqs, by_length);
    v[0] = x.start;
    v[1] = x.len;
    v[2] = x.row0;
    v[3] = w % a.Hq;
    return x.len > 0;
  };
  int item_no = 0, words[kItemWords] = {};
  auto tiles = [&](const SeqTile &x) {
    return x.len == 0 ? 0 : a.causal ? x.row0 / kTile + 1 : ceil_div(x.len, kTile);
  };

  if (warp == 0) {
    // -------------------------------------------------------- tile loads
    int it = 0, nq = 0;
    bool ok = true;
    while (ok && next_item<true>(ring, wait, item_no, lane, words)) {
      const SeqTile x{words[0], words[1], words[2]};
      [[maybe_unused]] const int h = words[3];
      const int n = tiles(x);
      ok = wait.all(q_empty, (nq & 1) ^ 1);
      if (!ok) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(q_full, 2 * L::tile_bytes);
        for (int j = 0; j < DP / 64; ++j) {
          load_box(sbase + j * kBoxBytes, &p.tq, 64 * j, h, x.start + x.row0, q_full);
          load_box(sbase + L::off_g + j * kBoxBytes, &p.tg, 64 * j, h, x.start + x.row0, q_full);
        }
      }
      __syncwarp();
      ++nq;
      for (int i = 0; i < n; ++i, ++it) {
        const int sk = it % kK, sv = it % kV;
        ok = wait.all(&k_empty[sk], ((it / kK) & 1) ^ 1);
        if (!ok) break;
        if (elect_one())
          load_tile<DP>(sbase + L::off_k + sk * L::tile_bytes, &p.tk, h / G, x.start + i * kTile,
                        &k_full[sk]);
        __syncwarp();
        ok = wait.all(&v_empty[sv], ((it / kV) & 1) ^ 1);
        if (!ok) break;
        if (elect_one())
          load_tile<DP>(sbase + L::off_v + sv * L::tile_bytes, &p.tv, h / G, x.start + i * kTile,
                        &v_full[sv]);
        __syncwarp();
      }
    }
    // every load has landed before the CTA may leave (after a wait that gave
    // up, a stage that was never filled may be waited for: bounded as well)
    if (nq) mbar_wait_bounded(q_full, (nq - 1) & 1, wait_limit, status);
    for (int i = max(it - kK, 0); i < it; ++i)
      mbar_wait_bounded(&k_full[i % kK], (i / kK) & 1, wait_limit, status);
    for (int i = max(it - kV, 0); i < it; ++i)
      mbar_wait_bounded(&v_full[i % kV], (i / kV) & 1, wait_limit, status);
    if (!ok) {  // a K tile loaded without its V tile
      mbar_wait_bounded(&k_full[it % kK], (it / kK) & 1, wait_limit, status);
    }
  } else if (warp == 1) {
    // -------------------------------------------------------- MMAs
    const int nk = (a.D + 15) / 16, no = nk * 16;
    int it = 0, nq = 0;  // key tiles and items so far
    bool ok = true;
    while (ok && next_item<false>(ring, wait, item_no, lane, words)) {
      const SeqTile x{words[0], words[1], words[2]};
      [[maybe_unused]] const int h = words[3];
      const int n = tiles(x);
      if (n == 0) continue;
      auto keys = [&](int i) {  // K of key tile i of this item has been loaded
        const int u = it + i;
        ok = wait.all(&k_full[u % kK], (u / kK) & 1);
      };
      auto values = [&](int i) {
        const int u = it + i;
        ok = wait.all(&v_full[u % kV], (u / kV) & 1);
      };
      auto scores = [&](int i) {  // S of key tile i
        const int u = it + i, s = u % kK;
        if (elect_one()) {
          mma_rows(tmem + (u & 1) * 128, sbase, sbase + L::off_k + s * L::tile_bytes, nk);
          mma_commit(&s_full[u & 1]);
        }
        __syncwarp();
      };
      auto grads = [&](int i) {  // do v^T of key tile i
        const int u = it + i, s = u % kV;
        if (elect_one()) {
          mma_rows(t_dp, sbase + L::off_g, sbase + L::off_v + s * L::tile_bytes, nk);
          mma_commit(dp_full);
          mma_commit(&v_empty[s]);
          if (i == n - 1) mma_commit(q_empty);  // the last use of this Q and dO
        }
        __syncwarp();
      };
      ok = wait.all(q_full, nq & 1);
      if (!ok) break;
      tc_fence_after();
      keys(0);
      if (ok) scores(0);
      if (ok) values(0);
      if (ok) grads(0);
      if (ok && n > 1) keys(1);
      if (ok && n > 1) scores(1);
      if (ok) ok = wait.all(acc_empty, (nq & 1) ^ 1);
      for (int i = 0; ok && i < n; ++i) {
        const int u = it + i, s = u % kK;
        // looked at while ds is formed, so that the queue below goes out at once
        if (i + 1 < n) values(i + 1);
        // (k_ready after the load, which came after the stage's last k_ready)
        if (ok && x.len - i * kTile < kTile) ok = wait.all(&k_ready[s], (u / kK) & 1);
        if (ok) ok = wait.all(&ds_ready[u & 1], (u >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if (i + 1 < n) grads(i + 1);
        if (elect_one()) {
          mma_halves(t_dq, tmem + (u & 1) * 128, sbase + L::off_k + s * L::tile_bytes, no, i != 0);
          mma_commit(&k_empty[s]);
        }
        __syncwarp();
        if (i + 2 < n) keys(i + 2);
        if (ok && i + 2 < n) scores(i + 2);
      }
      if (!ok) break;
      if (elect_one()) mma_commit(acc_full);
      __syncwarp();
      it += n;
      ++nq;
    }
    if (it || !ok) {  // every MMA issued has completed
      if (elect_one()) mma_commit(drain);
      __syncwarp();
      mbar_wait_bounded(drain, 0, wait_limit, status);
    }
  } else if (warp == 10) {
    // -------------------------------------------------------- K tiles' tails
    int it = 0;
    bool ok = true;
    while (ok && next_item<false>(ring, wait, item_no, lane, words)) {
      const SeqTile x{words[0], words[1], words[2]};
      [[maybe_unused]] const int h = words[3];
      const int n = tiles(x);
      for (int i = 0; i < n; ++i, ++it) {
        const int s = it % kK;
        ok = wait.all(&k_full[s], (it / kK) & 1);
        if (!ok) break;
        const int valid = x.len - i * kTile;
        if (valid < kTile) zero_rows<DP>(sm + L::off_k + s * L::tile_bytes, valid, lane);
        if (lane == 0) {
          mbar_arrive(&k_ready[s]);
          mbar_arrive(&k_empty[s]);
        }
        __syncwarp();
      }
    }
  } else if (warp < 10) {
    // -------------------------------------------------------- p and ds
    const int half = (warp - 2) >> 2, quarter = warp & 3;
    const int in_tile = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const float s2 = a.scale * kLog2E;
    int it = 0, nq = 0;
    bool ok = true;
    while (ok && next_item<false>(ring, wait, item_no, lane, words)) {
      const SeqTile x{words[0], words[1], words[2]};
      [[maybe_unused]] const int h = words[3];
      const int n = tiles(x);
      if (n == 0) continue;
      const int row = x.row0 + in_tile;
      const bool in = row < x.len;
      const int64_t at = (int64_t)h * a.T + x.start + row;
      const float lse2 = in ? a.lse[at] * kLog2E : 0.f, delta = in ? a.delta[at] : 0.f;
      const int last = a.causal ? min(row, x.len - 1) : x.len - 1;
      // by every row of this warp
      const int last_all = a.causal ? min(x.row0 + quarter * 32, x.len - 1) : x.len - 1;
      for (int i = 0; i < n; ++i, ++it) {
        const uint32_t ts = tmem + (it & 1) * 128 + 64 * half + lanes;
        ok = wait.all(&s_full[it & 1], (it >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        float2 pr[32];
        {
          uint32_t s[64];
          tmem_ld64(ts, s);
          const float2 sc = make_float2(s2, s2), off = make_float2(-lse2, -lse2);
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            float2 v = make_float2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1]));
            v = __ffma2_rn(v, sc, off);
            pr[c] = make_float2(ex2(v.x), ex2(v.y));
          }
        }
        const bool masked = i * kTile + 64 * half + 63 > last_all;
        ok = wait.all(dp_full, it & 1);
        if (!ok) break;
        tc_fence_after();
        uint32_t pk[32];
        {
          uint32_t d[64];
          tmem_ld64(t_dp + 64 * half + lanes, d);
          const float2 off = make_float2(-delta, -delta);
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float2 v = make_float2(__uint_as_float(d[2 * c]), __uint_as_float(d[2 * c + 1]));
            pr[c] = __fmul2_rn(pr[c], __fadd2_rn(v, off));
          }
          if (masked) {  // selected, not multiplied: what lies behind may be NaN
            const int lim = last - i * kTile - 64 * half;  // the last column seen
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              pr[c].x = 2 * c > lim ? 0.f : pr[c].x;
              pr[c].y = 2 * c + 1 > lim ? 0.f : pr[c].y;
            }
          }
#pragma unroll
          for (int c = 0; c < 32; ++c) pk[c] = pack_bf16(pr[c].x, pr[c].y);
        }
        __syncwarp();
        tmem_st32(ts, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ds_ready[it & 1]);
      }
      if (!ok) break;
      ok = wait.all(acc_full, nq & 1);
      if (!ok) break;
      ++nq;
      tc_fence_after();
      // this half's columns of dq
      constexpr int kCols = DP / 2;
      uint32_t v[kCols];
      __syncwarp();
      if constexpr (kCols == 64)
        tmem_ld64(t_dq + half * kCols + lanes, v);
      else
        tmem_ld32(t_dq + half * kCols + lanes, v);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty);
      if constexpr (kCols == 32) {
        uint32_t pk[16];
#pragma unroll
        for (int c = 0; c < 16; ++c)
          pk[c] = pack_bf16(__uint_as_float(v[2 * c]) * a.scale,
                            __uint_as_float(v[2 * c + 1]) * a.scale);
        const int r0 = x.row0 + quarter * 32;
        store_rows<32>(sm + L::off_stage + (warp - 2) * 2048, pk,
                       (bf16 *)a.dq + (int64_t)(x.start + r0) * a.ld_dq + (int64_t)h * a.D +
                           half * kCols,
                       a.ld_dq, x.len - r0, a.D - half * kCols, lane, &p.tdq, half * kCols, h,
                       x.start + r0);
      } else {
        if (in)
          store_half((bf16 *)a.dq + (int64_t)(x.start + row) * a.ld_dq + (int64_t)h * a.D +
                         half * kCols,
                     v, a.scale, min(kCols, a.D - half * kCols));
        __syncwarp();
      }
    }
    bulk_stores_done();
  } else {
    // -------------------------------------------------------- items
    ItemSource<decltype(find)> source(ring, wait, find, skipped ? -1 : (int)blockIdx.x, lane);
    bool ok = true;
    do {
      ok = source.publish(words);
    } while (ok && words[0] >= 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc1(tmem, 512);
  }
}

// ------------------------------------------------------------------- dk, dv

// One CTA: 128 key rows of one key head against the query tiles that see
// them, over all query heads of the group.  The score tile is transposed (rows
// are keys), so that p^T and ds^T stand in tensor memory as the left operands
// of p^T do and ds^T q.  Tensor memory: S^T, do v^T transposed, dv, dk.  Queue
// per query tile j: after p(j): dv += p do, S(j+1); after ds(j): dk += ds q,
// do v^T (j+1).
template <int DP> struct DkvLayout {
  static constexpr uint32_t tile_bytes = (DP / 64) * kBoxBytes;
  // Q stages (a Q tile is held from S to dk), dO stages, stages of row values
  static constexpr int kQ = DP == 128 ? 3 : 4, kG = DP == 128 ? 2 : 4, kR = 2;
  static constexpr uint32_t off_v = tile_bytes, off_q = 2 * tile_bytes;
  static constexpr uint32_t off_g = off_q + kQ * tile_bytes;
  static constexpr uint32_t off_row = off_g + kG * tile_bytes;  // [kR][-lse 128, -delta 128] floats
  static constexpr uint32_t off_bar = off_row + kR * 2 * kTile * 4;
  static constexpr uint32_t off_items =
      (off_bar + (2 * kQ + 2 * kG + 2 * kR + 8) * 8 + 16 + 15) / 16 * 16;
  static constexpr uint32_t off_order = off_items + ItemRing::kBytes;
  static constexpr uint32_t smem = off_order + SeqOrder::kBytes;
  static_assert(smem <= 227 * 1024, "shared memory per CTA");
};

template <int DP>
__global__ void __launch_bounds__(kBwdThreads, 1)
attn_dkv_tc(const __grid_constant__ BwdParams p, unsigned *status, long long wait_limit) {
  using L = DkvLayout<DP>;
  constexpr int kQ = L::kQ, kG = L::kG, kR = L::kR;
  // all of the 227 KB are spoken for, none is left to align the tiles by hand: the
  // declared alignment has to hold, and a kernel that finds it broken does nothing
  extern __shared__ __align__(1024) unsigned char smem_aligned[];
  unsigned char *sm = smem_aligned;
  const uint32_t sbase = smem_addr(sm);
  if ((sbase & 1023) != 0) {
    if (threadIdx.x == 0) atomicOr(status, kStatusSmemBase);
    pdl_wait();  // or the next kernel could start under the ones before this
    return;
  }
  float *rows = reinterpret_cast<float *>(sm + L::off_row);
  uint64_t *q_full = reinterpret_cast<uint64_t *>(sm + L::off_bar);
  uint64_t *q_empty = q_full + kQ, *g_full = q_empty + kQ, *g_empty = g_full + kG;
  uint64_t *s_full = g_empty + kG, *row_empty = s_full + kR;
  uint64_t *kv_full = row_empty + kR, *kv_empty = kv_full + 1;
  uint64_t *dp_full = kv_empty + 1, *p_ready = dp_full + 1, *ds_ready = p_ready + 1;
  uint64_t *acc_full = ds_ready + 1, *acc_empty = acc_full + 1, *drain = acc_empty + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const ItemRing ring(sm + L::off_items);
  const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kQ; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 2);  // the MMAs and the tail warp
    }
    for (int s = 0; s < kG; ++s) {
      mbar_init(&g_full[s], 1);
      mbar_init(&g_empty[s], 2);
    }
    for (int s = 0; s < kR; ++s) {
      mbar_init(&s_full[s], 2);  // the scores, and the row values with the tails' zeros
      mbar_init(&row_empty[s], kComputeWarps);
    }
    mbar_init(kv_full, 1);
    mbar_init(kv_empty, 1);
    mbar_init(dp_full, 1);
    mbar_init(p_ready, kComputeWarps);
    mbar_init(ds_ready, kComputeWarps);
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, kComputeWarps);
    mbar_init(drain, 1);
    ring.init(11);  // MMAs, eight compute warps, tails
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc1(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  const uint32_t t_dp = tmem + 128, t_dv = tmem + 256, t_dk = tmem + 256 + DP;
  const Waits wait{abort_flag, status, wait_limit};
  const AttnArgs &a = p.a;
  pdl_wait();
  pdl_trigger();
  const int G = a.Hq / a.Hkv;
  const bool skipped = attn_skipped(a.skip);
  SeqOrder seqs(sm + L::off_order);
  const bool by_length = a.B > 1 && a.B <= kSortMax;
  if (by_length && !skipped)
    seqs.make(a, reinterpret_cast<int *>(sm), [](int len) { return ceil_div(len, kTile); });
  // index w: share w % splits of the query heads of key head (w / splits) % Hkv;
  // tiles from the first one on, which most rows see
  const int shares = p.splits;
  auto find = [&](int w, int (&v)[kItemWords]) {
    const SeqTile x =
        tile_of(a, p.slots, w / (a.Hkv * shares), false, seqs, by_length);
    const int u = w % (a.Hkv * shares), c = u % shares;
    v[0] = x.start;
    v[1] = x.len;
    v[2] = x.row0;
    v[3] = u / shares;
    v[4] = c;
    v[5] = c * G / shares;        // its first head of the group, and how many
    v[6] = (c + 1) * G / shares - v[5];
    return x.len > 0;
  };
  int item_no = 0, words[kItemWords] = {};
  // query tiles first .. first + count - 1 of every head of the share; step j of
  // the item is query tile first + j % count of the share's head j / count
  auto first_tile = [&](const SeqTile &x) { return a.causal ? x.row0 / kTile : 0; };
  auto count = [&](const SeqTile &x) {
    return x.len == 0 ? 0 : ceil_div(x.len, kTile) - first_tile(x);
  };

  if (warp == 0) {
    // -------------------------------------------------------- tile loads
    int it = 0, nkv = 0;
    bool ok = true, half_step = false;
    while (ok && next_item<true>(ring, wait, item_no, lane, words)) {
      const SeqTile x{words[0], words[1], words[2]};
      [[maybe_unused]] const int hk = words[3], g0 = words[5], heads = words[6];
      const int nt = count(x), f = first_tile(x);
      ok = wait.all(kv_empty, (nkv & 1) ^ 1);
      if (!ok) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(kv_full, 2 * L::tile_bytes);
        for (int j = 0; j < DP / 64; ++j) {
          load_box(sbase + j * kBoxBytes, &p.tk, 64 * j, hk, x.start + x.row0, kv_full);
          load_box(sbase + L::off_v + j * kBoxBytes, &p.tv, 64 * j, hk, x.start + x.row0, kv_full);
        }
      }
      __syncwarp();
      ++nkv;
      for (int g = g0; ok && g < g0 + heads; ++g)
        for (int i = 0; i < nt; ++i, ++it) {
          const int sq = it % kQ, sg = it % kG, h = hk * G + g, row = x.start + (f + i) * kTile;
          ok = wait.all(&q_empty[sq], ((it / kQ) & 1) ^ 1);
          if (!ok) break;
          if (elect_one())
            load_tile<DP>(sbase + L::off_q + sq * L::tile_bytes, &p.tq, h, row, &q_full[sq]);
          __syncwarp();
          ok = wait.all(&g_empty[sg], ((it / kG) & 1) ^ 1);
          half_step = !ok;
          if (!ok) break;
          if (elect_one())
            load_tile<DP>(sbase + L::off_g + sg * L::tile_bytes, &p.tg, h, row, &g_full[sg]);
          __syncwarp();
        }
    }
    // every load has landed before the CTA may leave
    if (nkv) mbar_wait_bounded(kv_full, (nkv - 1) & 1, wait_limit, status);
    for (int i = max(it - kQ, 0); i < it; ++i)
      mbar_wait_bounded(&q_full[i % kQ], (i / kQ) & 1, wait_limit, status);
    for (int i = max(it - kG, 0); i < it; ++i)
      mbar_wait_bounded(&g_full[i % kG], (i / kG) & 1, wait_limit, status);
    if (half_step) mbar_wait_bounded(&q_full[it % kQ], (it / kQ) & 1, wait_limit, status);
  } else if (warp == 1) {
    // -------------------------------------------------------- MMAs
    const int nk = (a.D + 15) / 16, no = nk * 16;
    int it = 0, nkv = 0;
    bool ok = true;
    while (ok && next_item<false>(ring, wait, item_no, lane, words)) {
      const SeqTile x{words[0], words[1], words[2]};
      [[maybe_unused]] const int hk = words[3], g0 = words[5], heads = words[6];
      const int n = count(x) * heads;
      if (n == 0) continue;
      auto scores = [&](int j) {
        const int u = it + j, s = u % kQ;
        ok = wait.all(&q_full[s], (u / kQ) & 1);
        if (!ok) return;
        if (elect_one()) {
          mma_rows(tmem, sbase, sbase + L::off_q + s * L::tile_bytes, nk);
          mma_commit(&s_full[u % kR]);
        }
        __syncwarp();
      };
      auto outer = [&](int j) {  // dO of step j has been loaded
        const int u = it + j;
        ok = wait.all(&g_full[u % kG], (u / kG) & 1);
      };
      auto grads = [&](int j) {
        const int u = it + j, s = u % kG;
        if (elect_one()) {
          mma_rows(t_dp, sbase + L::off_v, sbase + L::off_g + s * L::tile_bytes, nk);
          mma_commit(dp_full);
          if (j == n - 1) mma_commit(kv_empty);  // the last use of this K and V
        }
        __syncwarp();
      };
      ok = wait.all(kv_full, nkv & 1);
      if (!ok) break;
      tc_fence_after();
      scores(0);
      if (ok) outer(0);
      if (ok) grads(0);
      if (ok) ok = wait.all(acc_empty, (nkv & 1) ^ 1);
      for (int j = 0; ok && j < n; ++j) {
        const int u = it + j, sq = u % kQ, sg = u % kG;
        // p is formed from the row values, so the tails of this step are zeroed
        ok = wait.all(p_ready, u & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) mma_halves(t_dv, tmem, sbase + L::off_g + sg * L::tile_bytes, no, j != 0);
        __syncwarp();
        if (j + 1 < n) scores(j + 1);
        if (ok && j + 1 < n) outer(j + 1);  // looked at while ds is formed
        if (ok) ok = wait.all(ds_ready, u & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          mma_commit(&g_empty[sg]);
          mma_halves(t_dk, t_dp, sbase + L::off_q + sq * L::tile_bytes, no, j != 0);
          mma_commit(&q_empty[sq]);
        }
        __syncwarp();
        if (j + 1 < n) grads(j + 1);
      }
      if (!ok) break;
      if (elect_one()) mma_commit(acc_full);
      __syncwarp();
      it += n;
      ++nkv;
    }
    if (it || !ok) {  // every MMA issued has completed
      if (elect_one()) mma_commit(drain);
      __syncwarp();
      mbar_wait_bounded(drain, 0, wait_limit, status);
    }
  } else if (warp == 10) {
    // ---------------------------- lse, delta, and the tails of the Q, dO tiles
    int it = 0;
    bool ok = true;
    while (ok && next_item<false>(ring, wait, item_no, lane, words)) {
      const SeqTile x{words[0], words[1], words[2]};
      [[maybe_unused]] const int hk = words[3], g0 = words[5], heads = words[6];
      const int nt = count(x), f = first_tile(x);
      for (int g = g0; ok && g < g0 + heads; ++g)
        for (int i = 0; i < nt; ++i, ++it) {
          const int sq = it % kQ, sg = it % kG, sr = it % kR, q0 = (f + i) * kTile;
          const int64_t at = (int64_t)(hk * G + g) * a.T + x.start + q0;
          float v[2][4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {  // in flight while the stage is waited for
            const int c = lane + 32 * e;
            const bool in = q0 + c < x.len;
            v[0][e] = in ? a.lse[at + c] * -kLog2E : 0.f;  // as the sums below take them
            v[1][e] = in ? -a.delta[at + c] : 0.f;
          }
          ok = wait.all(&row_empty[sr], ((it / kR) & 1) ^ 1) &&
               wait.all(&q_full[sq], (it / kQ) & 1) && wait.all(&g_full[sg], (it / kG) & 1);
          if (!ok) break;
          float *o = rows + sr * 2 * kTile;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            o[lane + 32 * e] = v[0][e];
            o[kTile + lane + 32 * e] = v[1][e];
          }
          const int valid = x.len - q0;
          if (valid < kTile) {
            zero_rows<DP>(sm + L::off_q + sq * L::tile_bytes, valid, lane);
            zero_rows<DP>(sm + L::off_g + sg * L::tile_bytes, valid, lane);
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&s_full[sr]);
            mbar_arrive(&q_empty[sq]);
            mbar_arrive(&g_empty[sg]);
          }
          __syncwarp();
        }
    }
  } else if (warp < 10) {
    // -------------------------------------------------------- p and ds
    const int half = (warp - 2) >> 2, quarter = warp & 3;
    const int in_tile = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t ts = tmem + 64 * half + lanes, td = t_dp + 64 * half + lanes;
    const float s2 = a.scale * kLog2E;
    int it = 0, nkv = 0;
    bool ok = true;
    while (ok && next_item<false>(ring, wait, item_no, lane, words)) {
      const SeqTile x{words[0], words[1], words[2]};
      [[maybe_unused]] const int hk = words[3], g0 = words[5], heads = words[6];
      const int nt = count(x), f = first_tile(x);
      if (nt == 0) continue;
      const int row = x.row0 + in_tile;  // key row within the sequence
      for (int j = 0; j < nt * heads; ++j, ++it) {
        const int sr = it % kR, q0 = (f + j % nt) * kTile + 64 * half;
        ok = wait.all(&s_full[sr], (it / kR) & 1);
        if (!ok) break;
        tc_fence_after();
        const float4 *lse = reinterpret_cast<const float4 *>(rows + sr * 2 * kTile + 64 * half);
        const float4 *delta = lse + kTile / 4;
        // columns lo .. hi - 1 of this half are queries that see this key
        const int lo = a.causal ? row - q0 : 0, hi = x.len - q0;
        const bool masked = (a.causal && q0 < x.row0 + quarter * 32 + 31) || hi < 64;
        float2 pr[32];
        {
          uint32_t v[64];
          tmem_ld64(ts, v);
          const float2 sc = make_float2(s2, s2);
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float4 l = lse[c];
            float2 x0 = make_float2(__uint_as_float(v[4 * c]), __uint_as_float(v[4 * c + 1]));
            float2 x1 = make_float2(__uint_as_float(v[4 * c + 2]), __uint_as_float(v[4 * c + 3]));
            x0 = __ffma2_rn(x0, sc, make_float2(l.x, l.y));
            x1 = __ffma2_rn(x1, sc, make_float2(l.z, l.w));
            pr[2 * c] = make_float2(ex2(x0.x), ex2(x0.y));
            pr[2 * c + 1] = make_float2(ex2(x1.x), ex2(x1.y));
          }
        }
        if (masked) {
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            pr[c].x = (2 * c < lo || 2 * c >= hi) ? 0.f : pr[c].x;
            pr[c].y = (2 * c + 1 < lo || 2 * c + 1 >= hi) ? 0.f : pr[c].y;
          }
        }
        uint32_t pk[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) pk[c] = pack_bf16(pr[c].x, pr[c].y);
        __syncwarp();
        tmem_st32(ts, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready);
        ok = wait.all(dp_full, it & 1);
        if (!ok) break;
        tc_fence_after();
        {
          uint32_t v[64];
          tmem_ld64(td, v);
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float4 d = delta[c];
            float2 x0 = make_float2(__uint_as_float(v[4 * c]), __uint_as_float(v[4 * c + 1]));
            float2 x1 = make_float2(__uint_as_float(v[4 * c + 2]), __uint_as_float(v[4 * c + 3]));
            pr[2 * c] = __fmul2_rn(pr[2 * c], __fadd2_rn(x0, make_float2(d.x, d.y)));
            pr[2 * c + 1] = __fmul2_rn(pr[2 * c + 1], __fadd2_rn(x1, make_float2(d.z, d.w)));
          }
          if (masked) {  // selected again: 0 times what lies behind may be NaN
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              pr[c].x = (2 * c < lo || 2 * c >= hi) ? 0.f : pr[c].x;
              pr[c].y = (2 * c + 1 < lo || 2 * c + 1 >= hi) ? 0.f : pr[c].y;
            }
          }
#pragma unroll
          for (int c = 0; c < 32; ++c) pk[c] = pack_bf16(pr[c].x, pr[c].y);
        }
        __syncwarp();
        tmem_st32(td, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(ds_ready);
          mbar_arrive(&row_empty[sr]);
        }
      }
      if (!ok) break;
      ok = wait.all(acc_full, nkv & 1);
      if (!ok) break;
      ++nkv;
      tc_fence_after();
      // the first group of warps stores dv, the second dk
      const uint32_t acc = (half ? t_dk : t_dv) + lanes;
      uint32_t v[DP / 64][64];
      __syncwarp();
#pragma unroll
      for (int j = 0; j < DP / 64; ++j) tmem_ld64(acc + 64 * j, v[j]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty);
      if (row < x.len && shares > 1) {
        float *o = p.part + (((int64_t)words[4] * 2 + (half ? 0 : 1)) * a.T + x.start + row) *
                                ((int64_t)a.Hkv * a.D) +
                   (int64_t)hk * a.D;
#pragma unroll
        for (int c = 0; c < DP; c += 4)
          if (c < a.D)
            *reinterpret_cast<uint4 *>(o + c) =
                make_uint4(v[c >> 6][c & 63], v[c >> 6][(c & 63) + 1], v[c >> 6][(c & 63) + 2],
                           v[c >> 6][(c & 63) + 3]);
      } else if (row < x.len) {
        bf16 *o = half ? (bf16 *)a.dk + (int64_t)(x.start + row) * a.ld_dk
                       : (bf16 *)a.dv + (int64_t)(x.start + row) * a.ld_dv;
        o += (int64_t)hk * a.D;
#pragma unroll
        for (int j = 0; j < DP / 64; ++j)
          store_half(o + 64 * j, v[j], half ? a.scale : 1.f, min(64, a.D - 64 * j));
      }
      __syncwarp();
    }
  } else {
    // -------------------------------------------------------- items
    ItemSource<decltype(find)> source(ring, wait, find, skipped ? -1 : (int)blockIdx.x, lane);
    bool ok = true;
    do {
      ok = source.publish(words);
    } while (ok && words[0] >= 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc1(tmem, 512);
  }
}

// Adds the shares of dk and dv in order, scales dk and rounds: eight columns of
// one row per thread, bound by L2, where the sums still are.  Rows of no
// sequence have no sums and are left alone.
__global__ void __launch_bounds__(256) attn_dkv_sum(const AttnArgs a, const float *part,
                                                    int shares) {
  pdl_wait();
  pdl_trigger();
  if (attn_skipped(a.skip)) return;
  const int64_t row = (int64_t)a.Hkv * a.D, packs = row / 8;
  const int64_t t0 = min(max(__ldg(a.cu), 0), (int)a.T);
  const int64_t t1 = min(max(__ldg(a.cu + a.B), 0), (int)a.T);
  const int64_t n = (t1 - t0) * packs * 2;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t u = i / packs, c = (i - u * packs) * 8;
    const int dv = (int)(u & 1);
    const int64_t t = t0 + (u >> 1);
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < shares; ++k) {
      const float4 *p =
          reinterpret_cast<const float4 *>(part + (((int64_t)k * 2 + dv) * a.T + t) * row + c);
      const float4 x = __ldcs(p), y = __ldcs(p + 1);
      s[0] += x.x;
      s[1] += x.y;
      s[2] += x.z;
      s[3] += x.w;
      s[4] += y.x;
      s[5] += y.y;
      s[6] += y.z;
      s[7] += y.w;
    }
    const float f = dv ? 1.f : a.scale;
    bf16 *o = (dv ? (bf16 *)a.dv + t * a.ld_dv : (bf16 *)a.dk + t * a.ld_dk) + c;
    *reinterpret_cast<uint4 *>(o) =
        make_uint4(pack_bf16(s[0] * f, s[1] * f), pack_bf16(s[2] * f, s[3] * f),
                   pack_bf16(s[4] * f, s[5] * f), pack_bf16(s[6] * f, s[7] * f));
  }
}

template <int DP>
cudaError_t launch(const AttnArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  BwdParams p;
  p.a = a;
  p.slots = (int)(a.T / kTile + a.B);
  p.splits = attn_bwd_splits(a.T, a.Hq, a.Hkv);
  p.part = attn_bwd_part(a);
  cudaError_t e = make_head_map(&p.tq, a.q, a.T, a.Hq, a.D, a.ld_q);
  if (e == cudaSuccess) e = make_head_map(&p.tk, a.k, a.T, a.Hkv, a.D, a.ld_k);
  if (e == cudaSuccess) e = make_head_map(&p.tv, a.v, a.T, a.Hkv, a.D, a.ld_v);
  if (e == cudaSuccess) e = make_head_map(&p.tg, a.do_, a.T, a.Hq, a.D, a.ld_do);
  if (e == cudaSuccess && DP == 64)
    e = make_head_map(&p.tdq, a.dq, a.T, a.Hq, a.D, a.ld_dq, 32, 32);
  unsigned *status = nullptr;
  if (e == cudaSuccess) e = device_status_ptr(dev, &status);
  if (e != cudaSuccess) return e;
  constexpr int kLanes = DP / 8;  // of a row of delta
  const int64_t blocks = ceil_div(a.T, (int64_t)(4 * 256 / kLanes)) * a.Hq;
  e = launch_pdl(attn_delta_packed<kLanes>, dim3((unsigned)blocks), dim3(256), 0, s, a);
  if (e != cudaSuccess) return e;
  constexpr size_t sq = DqLayout<DP>::smem, sk = DkvLayout<DP>::smem;
  blocks_per_sm((const void *)attn_dq_tc<DP>, kBwdThreads, sq, dev, 1);  // lifts the limits
  blocks_per_sm((const void *)attn_dkv_tc<DP>, kBwdThreads, sk, dev, 1);
  // one CTA per item
  e = launch_pdl(attn_dq_tc<DP>, dim3((unsigned)p.slots * (unsigned)a.Hq), dim3(kBwdThreads), sq, s,
                 p, status, kWaitLimitCycles);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn_dkv_tc<DP>, dim3((unsigned)p.slots * (unsigned)(a.Hkv * p.splits)),
                 dim3(kBwdThreads), sk, s, p, status, kWaitLimitCycles);
  if (e != cudaSuccess || p.splits == 1) return e;
  const int64_t want = ceil_div(a.T * a.Hkv * a.D * 2, (int64_t)(8 * 256));
  const int64_t most = (int64_t)dev.sms * 16;
  return launch_pdl(attn_dkv_sum, dim3((unsigned)(want < most ? want : most)), dim3(256), 0, s, a,
                    (const float *)p.part, p.splits);
}

}  // namespace

size_t attn_bwd_tc_workspace_bytes(int64_t T, int32_t Hq, int32_t Hkv, int32_t D) {
  const int n = attn_bwd_splits(T, Hq, Hkv);
  const size_t part = n > 1 ? (size_t)n * 2 * T * Hkv * D * sizeof(float) : 0;
  return delta_bytes(T, Hq) + part;
}

cudaError_t launch_attn_bwd_tc(const AttnArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  return a.D <= 64 ? launch<64>(a, dev, s) : launch<128>(a, dev, s);
}

}  // namespace ftk
