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
// the same keys.  12 warps:
//   warp 0      one lane issues the TMA tile loads: Q of the pair, then K and V
//               tiles through a ring of kStages;
//   warps 1,11  one lane each issues the MMAs of tile 0 and 1 (S = Q K^T from
//               shared memory; O += P V with P read from tensor memory);
//   warps 2-5   softmax of tile 0, one query row per thread (no shuffles),
//   warps 6-9   and of tile 1;
//   warp 10     finds the work items, and zeroes the rows of a V tile that lie
//               behind its sequence's end before the MMAs may read them.
// A key tile's 128 scores are taken as two halves of 64, each a step of the
// running softmax of its own: the first half's P V runs while the second
// half's exponentials are formed.  Within a half the exponentials do not wait
// for the maximum: they are formed against the one that stands, the half's own
// maximum beside them, and only if some row passes the standing one by more
// than 2^kRaise are they formed again, after O and l of the rows that passed
// were brought to the new maximum: 347 against 374 us with the maximum first
// (one causal sequence of 8,192 tokens, 32/8 x 128).  Each row goes by its own
// scores alone, so its bits do not depend on its neighbours in the tile, and
// rows behind a sequence's end start nothing.  Keeping a lower maximum changes
// nothing in exact arithmetic (o and l carry the same factor) and keeps p <=
// 2^kRaise.  Rounding p to bf16 (2^-8 relative at most, per term) is the price
// of the tensor cores' second product.
// Tensor memory: S0 S1 (128 columns each), O0 O1.  P, in bf16, replaces the
// scores it came from; with head sizes up to 64 there is room for P beside S,
// and the next scores are formed while the current ones are still worked on.
// Measured, one causal sequence of 32,768 tokens, 64/8 heads of 128: 11.7 ms, 1.51
// PFLOP/s over the unmasked scores (0.87 of what a library GEMM sustains); of
// 8,192, 32/8: 347 us with heads of 128 (tensor pipe busy 69% of the cycles, the
// bound), 242 with heads of 64 (49%; the exponentials' unit 49%, issue 56%);
// 16,384 tokens in 85 sequences, 14/2 x 64: 47 us, mostly the start and end of
// items of one or two key tiles.  Masks looked at by each warp's own rows and O
// leaving by tile stores were worth 15 and 2 us of the last two.
#include <cmath>

#include "attn_tc.cuh"

namespace ftk {

namespace attn {

cudaError_t make_head_map(CUtensorMap *map, const void *base, int64_t T, int64_t H, int64_t D,
                          int64_t ld, uint32_t rows, uint32_t cols) {
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)ld * 2};
  const cuuint32_t box[3] = {cols, 1, rows};
  return tc::encode_bf16_map(map, base, 3, dims, strides, box,
                             cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

}  // namespace attn

namespace {

using namespace attn;

constexpr int kFwdThreads = 384;
constexpr float kRaise = 8.f;

struct FwdParams {
  CUtensorMap tq, tk, tv, to;
  AttnArgs a;
  int nslots;  // pair slots per key head
};

// Two query tiles of one key head: heads h[], first rows row0[] (within the
// sequence) and key tiles n[] each (0: no such tile).
struct FwdItem {
  int start, len, hk;
  int h[2], row0[2], n[2];
  __device__ __forceinline__ int tiles() const { return max(n[0], n[1]); }
  __device__ __forceinline__ FwdItem() {}
  __device__ __forceinline__ explicit FwdItem(const int (&v)[kItemWords])
      : start(v[0]), len(v[1]), hk(v[2]) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      h[t] = v[3 + t];
      row0[t] = v[5 + t];
      n[t] = v[7 + t];
    }
  }
  __device__ __forceinline__ void to(int (&v)[kItemWords]) const {
    v[0] = start;
    v[1] = len;
    v[2] = hk;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      v[3 + t] = h[t];
      v[5 + t] = row0[t];
      v[7 + t] = n[t];
    }
    v[9] = v[10] = v[11] = 0;
  }
};

// Halves of key tile i that hold keys: only a sequence's last tile may have one.
__device__ __forceinline__ int halves_of(const FwdItem &x, int i) {
  return x.len - i * kTile > 64 ? 2 : 1;
}

// Pairs of (row tile, head of the group) of one sequence: the slots of
// attn_common.cuh with floor((slot G + 1) / 2) + b in place of the slot.
__device__ __forceinline__ int pair_base(int c, int b, int G) {
  return ((max(c, 0) / kTile + b) * G + 1) / 2 + b;
}

__device__ __forceinline__ int pairs_of(int len, int G) {
  return (ceil_div(len, kTile) * G + 1) / 2;
}

// Item `item`: key heads fastest, then the pairs in the order of their slots or
// by the length of their sequence.  Within a sequence from the last pair back,
// whose rows see most keys.
__device__ __forceinline__ FwdItem fwd_item(const AttnArgs &a, int nslots, int item,
                                            const SeqOrder &seqs, bool by_length) {
  FwdItem w;
  const int G = a.Hq / a.Hkv;
  w.hk = item % a.Hkv;
  int b, pair = 0;
  if (by_length) {
    const int u = item / a.Hkv, r = u < seqs.total ? seqs.rank_of(u, a.B) : 0;
    b = seqs.order[r];
    pair = u < seqs.total ? u - seqs.base[r] : 1 << 30;
  } else {
    const int slot = nslots - 1 - item / a.Hkv;
    int lo = 1, hi = a.B;
    while (lo <= hi) {
      const int mid = (lo + hi) >> 1;
      if (pair_base(__ldg(a.cu + mid), mid, G) <= slot)
        lo = mid + 1;
      else
        hi = mid - 1;
    }
    b = min(lo - 1, a.B - 1);
    pair = slot;
  }
  const int c0 = min(max(__ldg(a.cu + b), 0), (int)a.T);
  const int c1 = min(max(__ldg(a.cu + b + 1), c0), (int)a.T);
  w.start = c0;
  w.len = c1 - c0;
  const int nt = ceil_div(w.len, kTile);
  const int64_t f0 = 2 * (by_length ? (int64_t)pairs_of(w.len, G) - 1 - pair
                                    : (int64_t)pair - pair_base(c0, b, G));
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
  static constexpr int kStages = DP == 128 ? 4 : 8;
  static constexpr uint32_t off_ring = 2 * tile_bytes;
  static constexpr uint32_t off_stage = off_ring + kStages * tile_bytes;  // 4 KB per softmax warp
  static constexpr uint32_t off_bar = off_stage + 8 * 4096;
  static constexpr uint32_t off_items = (off_bar + (3 * kStages + 20) * 8 + 16 + 15) / 16 * 16;
  static constexpr uint32_t off_order = off_items + ItemRing::kBytes;
  static constexpr uint32_t smem = off_order + SeqOrder::kBytes + 1024;
  static_assert(smem <= 227 * 1024, "shared memory per CTA");
};

template <int DP>
__global__ void __launch_bounds__(kFwdThreads, 1)
attn_fwd_tc(const __grid_constant__ FwdParams p, unsigned *status, long long wait_limit) {
  using L = FwdLayout<DP>;
  constexpr int kStages = L::kStages;
  constexpr bool kApart = DP <= 64;  // P beside S in tensor memory, not over it
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
  // p_full and o_full per [tile][half]: with one barrier for both halves, the
  // second could complete before the other side looked for the first
  uint64_t *o_full = p_full + 4;
  uint64_t *o_empty = o_full + 4;
  uint64_t *s_read = o_empty + 2;
  uint64_t *drain = s_read + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 2);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const ItemRing ring(sm + L::off_items);
  const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 3);  // both MMA warps and the tail warp
      mbar_init(&v_ready[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 1);
      mbar_init(&q_empty[t], 1);
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[2 * t], 4);
      mbar_init(&p_full[2 * t + 1], 4);
      mbar_init(&o_full[2 * t], 1);
      mbar_init(&o_full[2 * t + 1], 1);
      mbar_init(&o_empty[t], 4);
      mbar_init(&s_read[t], 4);
      mbar_init(&drain[t], 1);
    }
    ring.init(11);  // loads, MMAs of both tiles, eight softmax warps
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc1(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  const Waits wait{abort_flag, status, wait_limit};
  const AttnArgs &a = p.a;
  pdl_wait();
  pdl_trigger();
  const bool skipped = attn_skipped(a.skip);
  int item_no = 0, words[kItemWords];
  SeqOrder seqs(sm + L::off_order);
  const bool by_length = a.B > 1 && a.B <= kSortMax;
  if (by_length && !skipped)
    seqs.make(a, reinterpret_cast<int *>(sm), [&](int len) { return pairs_of(len, a.Hq / a.Hkv); });

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
    while (ok && next_item<true>(ring, wait, item_no, lane, words)) {
      const FwdItem x(words);
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
#pragma unroll
    for (int t = 0; t < 2; ++t)
      if (nq[t]) mbar_wait_bounded(&q_full[t], (nq[t] - 1) & 1, wait_limit, status);
    for (int i = max(it - kStages, 0); i < it; ++i)
      mbar_wait_bounded(&kv_full[i % kStages], (i / kStages) & 1, wait_limit, status);
  } else if (warp == 1 || warp == 11) {
    // -------------------------------------------------------- MMAs of tile t
    const int t = warp == 11;
    const int nk = (a.D + 15) / 16, no = nk * 16;  // contraction steps of S, columns of O
    const uint32_t t_s = tmem + t * 128, t_o = tmem + 256 + t * DP;
    const uint32_t t_p = kApart ? tmem + 384 + t * 64 : t_s;
    int it = 0, nq = 0, ns = 0;  // ring entries, items, score tiles so far
    int np0 = 0, np1 = 0;        // first and second halves so far
    bool ok = true;
    while (ok && next_item<false>(ring, wait, item_no, lane, words)) {
      const FwdItem x(words);
      const int n = x.tiles(), mine = t ? x.n[1] : x.n[0];
      if (n == 0) continue;
      auto keys = [&](int e) {  // ring entry e has been loaded
        const int s = e % kStages;
        ok = wait.all(&kv_full[s], (e / kStages) & 1);
      };
      // scores of key tile i, whose keys (loaded) are ring entry e
      auto scores = [&](int i, int e) {
        const int s = e % kStages;
        if (kApart && i > 0) {  // the scores before these have been read
          ok = wait.all(&s_read[t], (ns - 1) & 1);
          if (!ok) return;
        }
        tc_fence_after();
        if (elect_one()) {
          mma_rows(t_s, sbase + t * L::tile_bytes, sbase + L::off_ring + s * L::tile_bytes, nk);
          mma_commit(&s_full[t]);
          mma_commit(&kv_empty[s]);
          if (i == mine - 1) mma_commit(&q_empty[t]);  // the last use of this Q tile
        }
        __syncwarp();
        ++ns;
      };
      auto pass = [&](int e) {  // an entry of the other tile's alone
        keys(e);
        if (ok && lane == 0) mbar_arrive(&kv_empty[e % kStages]);
        __syncwarp();
      };
      if (mine) {
        ok = wait.all(&q_full[t], nq & 1);
        if (ok) keys(it);
        if (ok) scores(0, it);
      } else {
        pass(it);
      }
      for (int i = 0; ok && i < n; ++i) {
        const int ev = it + 2 * i + 1, sv = ev % kStages;  // V of this tile; K of the next follows
        const bool next = i + 1 < mine;
        if (i >= mine) {
          pass(ev);
          if (ok && i + 1 < n) pass(ev + 1);
          continue;
        }
        if (kApart && next) {  // the next scores run under this tile's exponentials
          keys(ev + 1);
          if (ok) scores(i + 1, ev + 1);
          if (!ok) break;
        }
        keys(ev);
        // after the load, which came after kv_empty of the stage's last use, hence
        // after that use's v_ready: this wait sees no older phase
        if (ok && x.len - i * kTile < kTile) ok = wait.all(&v_ready[sv], (ev / kStages) & 1);
        if (!ok) break;
        const int halves = halves_of(x, i);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // with room beside S the softmax hands over a tile's p at once
          if (h == halves) break;
          if (!kApart || h == 0) ok = wait.all(&p_full[2 * t + h], (h ? np1 : np0) & 1);
          if (ok && i == 0 && h == 0) ok = wait.all(&o_empty[t], (nq & 1) ^ 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            mma_half(t_o, t_p + h * (kApart ? 32 : 64), sbase + L::off_ring + sv * L::tile_bytes, h,
                     no, i != 0 || h != 0);
            if (!kApart || h == halves - 1) mma_commit(&o_full[kApart ? 2 * t : 2 * t + h]);
            if (h == halves - 1) mma_commit(&kv_empty[sv]);
          }
          __syncwarp();
          np0 += h == 0;
          np1 += h;
          if (!kApart && h == 0 && next) {  // looked at while the second half is formed
            keys(ev + 1);
            if (!ok) break;
          }
        }
        if (!ok) break;
        if (!kApart && next) scores(i + 1, ev + 1);
        if (ok && !next && i + 1 < n) pass(ev + 1);
      }
      it += 2 * n;
      nq += mine != 0;
    }
    if (ns) {  // every MMA issued has completed
      if (elect_one()) mma_commit(&drain[t]);
      __syncwarp();
      mbar_wait_bounded(&drain[t], 0, wait_limit, status);
    }
  } else if (warp == 10) {
    // -------------------------------------------------------- items, V tiles' tails
    auto find = [&](int index, int (&v)[kItemWords]) {
      const FwdItem x = fwd_item(a, p.nslots, index, seqs, by_length);
      x.to(v);
      return x.tiles() > 0;
    };
    ItemSource<decltype(find)> source(ring, wait, find, skipped ? -1 : (int)blockIdx.x, lane);
    int it = 0;
    bool ok = source.publish(words);
    while (ok && words[0] >= 0) {
      const FwdItem x(words);
      const int n = x.tiles();
      for (int i = 0; ok && i < 2 * n; ++i, ++it) {  // K0 V0 K1 V1 ..., as loaded
        const int s = it % kStages;
        ok = wait.all(&kv_full[s], (it / kStages) & 1);
        if (!ok) break;
        const int valid = x.len - (i >> 1) * kTile;
        if ((i & 1) && valid < kTile)
          zero_rows<DP>(sm + L::off_ring + s * L::tile_bytes, valid, lane);
        if (lane == 0) {
          mbar_arrive(&v_ready[s]);  // before kv_empty: see the MMA warps' wait
          mbar_arrive(&kv_empty[s]);
        }
        __syncwarp();
      }
      if (ok) ok = source.publish(words);
    }
  } else if (warp < 10) {
    // -------------------------------------------------------- softmax
    const int t = (warp - 2) >> 2, quarter = warp & 3;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t ts = tmem + t * 128 + lanes, to = tmem + 256 + t * DP + lanes;
    const uint32_t tp = kApart ? tmem + 384 + t * 64 + lanes : ts;
    const float s2 = a.scale * kLog2E;
    const float2 sc = make_float2(s2, s2);
    int ns = 0, np0 = 0, np1 = 0;  // score tiles, first and second halves so far
    bool ok = true;
    while (ok && next_item<false>(ring, wait, item_no, lane, words)) {
      const FwdItem x(words);
      // selected, not indexed: an index would put the item into local memory,
      // and beside this much shared memory L1 holds next to nothing of it
      const int n = t ? x.n[1] : x.n[0], row0 = t ? x.row0[1] : x.row0[0];
      const int head = t ? x.h[1] : x.h[0];
      if (n == 0) continue;
      const int row = row0 + quarter * 32 + lane;                   // within the sequence
      const bool in = row < x.len;  // behind it: rows of another sequence, or of none
      // rows behind the end start no raise (a limit in a register: as a term of the vote,
      // `in` cost 3% with heads of 128)
      const float limit = in ? kRaise : INFINITY;
      const int last = a.causal ? min(row, x.len - 1) : x.len - 1;  // the last key seen
      // by every row of this warp, and by any
      const int last_all = a.causal ? min(row0 + quarter * 32, x.len - 1) : x.len - 1;
      const int last_any = a.causal ? row0 + quarter * 32 + 31 : x.len - 1;
      float m = -INFINITY, ms = 0.f;
      float2 l2 = make_float2(0.f, 0.f);
      for (int i = 0; ok && i < n; ++i, ++ns) {
        ok = wait.all(&s_full[t], ns & 1);
        if (!ok) break;
        tc_fence_after();
        const int halves = halves_of(x, i);
        // of a tile on the diagonal the first two warps see nothing of its second half
        // (left out with heads of up to 64; with the steps of half a tile the branch
        // costs more than it saves, 371 against 347 us)
        [[maybe_unused]] const bool two = halves == 2 && i * kTile + 64 <= last_any;
        // 64 columns from column 64 h on, masked
        auto load = [&](int h, uint32_t (&s)[64]) {
          __syncwarp();
          tmem_ld64(ts + 64 * h, s);
          const int c0 = i * kTile + 64 * h;
          if (c0 + 63 > last_all) {
            const int lim = last - c0;
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (c > lim) s[c] = 0xff800000u;  // -inf
          }
        };
        auto highest = [&](const uint32_t (&s)[64]) {
          float mx[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mx[e] = fmaxf(__uint_as_float(s[e]), __uint_as_float(s[e + 4]));
#pragma unroll
          for (int c = 8; c < 64; c += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mx[e] = max3(mx[e], __uint_as_float(s[c + e]), __uint_as_float(s[c + e + 4]));
          return fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
        };
        // p against the standing maximum: 32 words of bf16 pairs, and their sum
        auto probs = [&](const uint32_t (&s)[64], uint32_t (&pk)[32]) {
          const float2 off = make_float2(-ms, -ms);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < 64; c += 2) {
            float2 v = make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1]));
            v = __ffma2_rn(v, sc, off);
            v.x = ex2(v.x);
            v.y = ex2(v.y);
            sum[(c >> 1) & 1] = __fadd2_rn(sum[(c >> 1) & 1], v);
            pk[c >> 1] = pack_bf16(v.x, v.y);
          }
          return __fadd2_rn(sum[0], sum[1]);
        };
        // brings O and l from the standing maximum to `to_m`, once the P V that
        // `bar` counts is in O; f is 1 exactly in the rows that keep theirs
        auto raise = [&](float to_m, uint64_t *bar, int count) {
          const float nm = to_m == -INFINITY ? 0.f : to_m * s2;
          const float f = to_m == m ? 1.f : ex2(m * s2 - nm);
          ok = wait.all(bar, (count - 1) & 1);
          if (!ok) return;
          tc_fence_after();
          __syncwarp();
#pragma unroll 1
          for (int c = 0; c < DP; c += 16) {
            uint32_t o[16];
            tmem_ld16(to + c, o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st16(to + c, o);
          }
          l2.x *= f;
          l2.y *= f;
          m = to_m;
          ms = nm;
        };
        if constexpr (kApart) {
          uint32_t s[64], p0[32], p1[32];
          load(0, s);
          float top = highest(s);
          if (i == 0) {
            m = top;
            ms = m == -INFINITY ? 0.f : m * s2;
          }
          float2 sum = probs(s, p0);
          if (two) {
            load(1, s);
            top = fmaxf(top, highest(s));
          }
          const bool passed = (top - m) * s2 > limit;
          if (__any_sync(0xffffffffu, passed)) {
            if (i > 0) {
              raise(passed ? top : m, &o_full[2 * t], np0);
              if (!ok) break;
            } else {  // nothing in O yet: the first half's maximum was too low
              m = passed ? top : m;
              ms = m == -INFINITY ? 0.f : m * s2;
            }
            load(0, s);
            sum = probs(s, p0);
            if (two) load(1, s);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_read[t]);  // the next scores may replace these
          if (two) {
            sum = __fadd2_rn(sum, probs(s, p1));
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) p1[c] = 0u;
          }
          l2 = __fadd2_rn(l2, sum);
          if (np0 > 0) {  // the last P V has read P's columns
            ok = wait.all(&o_full[2 * t], (np0 - 1) & 1);
            if (!ok) break;
            tc_fence_after();
          }
          __syncwarp();
          tmem_st32(tp, p0);
          if (halves == 2) tmem_st32(tp + 32, p1);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * t]);
          ++np0;
        } else {
#pragma unroll 1
          for (int h = 0; h < halves; ++h) {
            uint32_t s[64], pk[32];
            load(h, s);
            const float top = highest(s);
            if (i == 0 && h == 0) {
              m = top;
              ms = m == -INFINITY ? 0.f : m * s2;
            }
            float2 sum = probs(s, pk);
            const float to_m = (top - m) * s2 > limit ? top : m;
            if (__any_sync(0xffffffffu, to_m > m)) {
              // (never the first half of the first tile, which set the maximum)
              raise(to_m, &o_full[2 * t + 1 - h], h ? np0 : np1);
              if (!ok) break;
              sum = probs(s, pk);
            }
            l2 = __fadd2_rn(l2, sum);
            __syncwarp();
            tmem_st32(tp + 64 * h, pk);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[2 * t + h]);
            np0 += h == 0;
            np1 += h;
          }
        }
      }
      if (!ok) break;
      ok = !kApart && halves_of(x, n - 1) == 2 ? wait.all(&o_full[2 * t + 1], (np1 - 1) & 1)
                                    : wait.all(&o_full[2 * t], (np0 - 1) & 1);
      if (!ok) break;
      tc_fence_after();
      const float l = l2.x + l2.y, inv = 1.f / l;
      bf16 *o = (bf16 *)a.o + (int64_t)(x.start + row0 + quarter * 32) * a.ld_o +
                (int64_t)head * a.D;
      // all columns first, the warp converged, then the divergent stores: a
      // tensor-memory load must never sit behind a branch that lanes take apart
      uint32_t v[DP / 64][64];
      __syncwarp();
#pragma unroll
      for (int j = 0; j < DP / 64; ++j) tmem_ld64(to + 64 * j, v[j]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_empty[t]);  // the next pair's O may be written
#pragma unroll
      for (int j = 0; j < DP / 64; ++j) {
        uint32_t pk[32];
#pragma unroll
        for (int c = 0; c < 32; ++c)
          pk[c] = pack_bf16(__uint_as_float(v[j][2 * c]) * inv,
                            __uint_as_float(v[j][2 * c + 1]) * inv);
        store_rows<64>(sm + L::off_stage + (warp - 2) * 4096, pk, o + 64 * j, a.ld_o,
                       x.len - row0 - quarter * 32, a.D - 64 * j, lane, &p.to, 64 * j, head,
                       x.start + row0 + quarter * 32);
      }
      if (in && a.lse)
        a.lse[(int64_t)head * a.T + x.start + row] = ms * kLn2 + logf(l);
      __syncwarp();
    }
    bulk_stores_done();
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
  if (e == cudaSuccess) e = make_head_map(&p.to, a.o, a.T, a.Hq, a.D, a.ld_o, 32);
  unsigned *status = nullptr;
  if (e == cudaSuccess) e = device_status_ptr(dev, &status);
  if (e != cudaSuccess) return e;
  constexpr size_t smem = FwdLayout<DP>::smem;
  blocks_per_sm((const void *)attn_fwd_tc<DP>, kFwdThreads, smem, dev, 1);  // lifts the limit
  const unsigned grid = (unsigned)p.nslots * (unsigned)a.Hkv;  // one CTA per item
  return launch_pdl(attn_fwd_tc<DP>, dim3(grid), dim3(kFwdThreads), smem, s, p, status,
                    kWaitLimitCycles);
}

}  // namespace

cudaError_t launch_attn_fwd_tc(const AttnArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  return a.D <= 64 ? launch<64>(a, dev, s) : launch<128>(a, dev, s);
}

}  // namespace ftk
