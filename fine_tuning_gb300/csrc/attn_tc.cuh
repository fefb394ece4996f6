// Tensor-core pieces shared by the attention kernels (attn_fwd_tc.cu,
// attn_bwd_tc.cu): single-CTA tcgen05 instructions, tile loads, descriptors
// of the staged tiles, tensor-memory loads and stores, bounded waits.
//
// Every operand tile is kTile = 128 rows (tokens) of one head, staged as boxes
// of 64 columns: 128 rows x 128 bytes with the 128-byte swizzle, 16 KB each,
// box j at j x 16 KB.  The same bytes serve as a K-major operand (rows = M or
// N, the head's columns contracted) and as an MN-major one (columns = N, the
// rows contracted), so no tile is ever transposed or staged twice.
#pragma once

#include "attn_common.cuh"
#include "tc_gemm.cuh"

namespace ftk {
namespace attn {

using tc::elect_one;
using tc::tc_fence_after;
using tc::tc_fence_before;
using tc::tmem_ld32;
using tc::tmem_ld64;

// Bit of the device status word beside kStatusWaitTimeout: shared memory began off
// the tiles' alignment.
constexpr unsigned kStatusSmemBase = 2u;

constexpr int kTile = 128;
constexpr uint32_t kBoxBytes = kTile * 128;  // 64 bf16 columns of a tile

// One tensor [T, H, D] read in boxes of 128 tokens x one head x 64 columns;
// columns past D and tokens past T read as zeros.  rows, cols: tokens and columns
// of a box (64 columns with the 128-byte swizzle, 32 with the 64-byte one).
cudaError_t make_head_map(CUtensorMap *map, const void *base, int64_t T, int64_t H, int64_t D,
                          int64_t ld, uint32_t rows = kTile, uint32_t cols = 64);

__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, int col, int head,
                                         int row, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(col), "r"(head), "r"(row), "r"(smem_addr(bar))
      : "memory");
}

// A whole tile: DP / 64 boxes.
template <int DP>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap *map, int head, int row,
                                          uint64_t *bar) {
  mbar_arrive_expect_tx(bar, (DP / 64) * kBoxBytes);
#pragma unroll
  for (int j = 0; j < DP / 64; ++j) load_box(dst + j * kBoxBytes, map, 64 * j, head, row, bar);
}

__device__ __forceinline__ void tmem_alloc1(uint32_t *slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_addr(slot)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc1(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}

// v, which every lane of the warp holds, in a form that the compiler knows to
// be one value per warp (the reduction's result is a uniform register).  The
// MMAs and tile loads take their operands from uniform registers: values that
// only happen to be equal are moved there one by one before each of them.
__device__ __forceinline__ int uniform(int v) { return __reduce_max_sync(0xffffffffu, v); }
__device__ __forceinline__ uint32_t uniform(uint32_t v) {
  return __reduce_max_sync(0xffffffffu, v);
}

// D [128 x N] (+)= A B^T, A and B in shared memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// The same with A in tensor memory: row i in lane i, two bf16 per column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives once on bar when this thread's earlier MMAs have completed.
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_addr(bar))
      : "memory");
}

// Instruction descriptor, kind::f16, M = 128: D fp32, A and B bf16.
__device__ __forceinline__ uint32_t idesc_of(int n, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(kTile >> 4) << 24);
}
// K-major operand, contraction step kk of 16 columns: box kk / 4, 32 bytes per step.
__device__ __forceinline__ uint64_t desc_k(uint32_t tile, int kk) {
  return tc::desc_sw128(tile + (uint32_t)(kk >> 2) * kBoxBytes + (uint32_t)(kk & 3) * 32u);
}
// MN-major operand, contraction step kk of 16 rows; 64-column blocks kBoxBytes
// apart (leading byte offset), 8-row swizzle atoms 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_mn(uint32_t tile, int kk) {
  const uint32_t addr = tile + (uint32_t)kk * (16u * 128u);
  return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)(kBoxBytes >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// acc [128 x 128] = A B^T over nk steps of 16 columns (both tiles K-major).
__device__ __forceinline__ void mma_rows(uint32_t acc, uint32_t a, uint32_t b, int nk) {
  const uint32_t id = idesc_of(kTile, false);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    if (kk < nk) mma_ss(acc, desc_k(a, kk), desc_k(b, kk), id, kk != 0);
}
// acc [128 x n] (+)= P B over rows 64 half .. 64 half + 63 of B; P [128 x 64] of
// that half in bf16 in 32 columns of tensor memory from p on.
__device__ __forceinline__ void mma_half(uint32_t acc, uint32_t p, uint32_t b, int half, int n,
                                         bool accumulate) {
  const uint32_t id = idesc_of(n, true);
#pragma unroll
  for (int kk = 0; kk < 4; ++kk)
    mma_ts(acc, p + (uint32_t)kk * 8u, desc_mn(b, 4 * half + kk), id, accumulate || kk != 0);
}

// The larger of three (one instruction).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 16 or 32 columns of this thread's lane from registers.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
      "%29, %30, %31, %32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
      "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]),
      "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]),
      "r"(v[30]), "r"(v[31])
      : "memory");
}
// 16 columns of this thread's lane, waited for in the same statement.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// 2^x by the hardware approximation (relative error about 2^-22, 2^-inf = +0).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// One look at a barrier that may suspend the warp for up to about a
// millisecond.  A wait that spins instead takes issue slots and shared-memory
// queue entries (which the exponentials go through as well) from the warps
// that work.
__device__ __forceinline__ bool mbar_try_wait_long(uint64_t *bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity), "r"(1000000)
      : "memory");
  return done != 0;
}

// The waits of a CTA: bounded, and over as soon as any role has given up.
struct Waits {
  volatile int *abort;
  unsigned *status;
  long long limit;
  __device__ __forceinline__ bool within(uint64_t *bar, uint32_t parity, long long cycles) const {
    if (mbar_try_wait_long(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait_long(bar, parity)) {
      if (*abort) return false;
      if (clock64() - t0 > cycles) {
        atomicOr(status, kStatusWaitTimeout);
        *abort = 1;
        return false;
      }
    }
    return true;
  }
  // for a whole warp that goes on together or stops together
  __device__ __forceinline__ bool all(uint64_t *bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, within(bar, parity, limit));
  }
  // The same for a wait that lasts as long as another role of this CTA works on a
  // whole item, or searches for one: dk and dv of 128 heads that share one, over 1M
  // tokens, are 1M tile steps of some 2,260 cycles.  What that role waits for is
  // bounded by `limit`, tile by tile, and its giving up ends this wait too; the
  // bound here (a quarter of an hour) is only the last resort.
  __device__ __forceinline__ bool all_item(uint64_t *bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, within(bar, parity, limit << 10));
  }
};

// ------------------------------------------------------------- work items
//
// The grid has one CTA per item (a tile, or pair of tiles, and a head), but as
// many run as fit, and each goes on to the items of CTAs that have not started
// yet (cluster launch control: a running CTA cancels the launch of a waiting
// one and takes its index over).  So items of very different lengths even out
// without a counter in memory that calls on two streams would share.
//
// One warp of the CTA asks for the next item when the loading warp has no
// more to load for the current one (an item asked for earlier would be tied to
// this CTA while others run dry: with a few long items per SM that cost 19%),
// finds its sequence and tile once for all roles, and hands it over in a ring
// of two slots; empty items are dropped there.
constexpr int kItemWords = 12;

struct ItemRing {
  uint64_t *want;   // the loading warp is done with the last item
  uint64_t *asked;  // the answer has arrived (16 bytes)
  uint64_t *full;   // [2]
  uint64_t *empty;  // [2]
  int *slots;       // [2][kItemWords]
  uint4 *answer;
  static constexpr uint32_t kBytes = 16 + 2 * kItemWords * 4 + 6 * 8;  // from a multiple of 16

  __device__ __forceinline__ explicit ItemRing(unsigned char *at) {
    answer = reinterpret_cast<uint4 *>(at);
    slots = reinterpret_cast<int *>(at + 16);
    asked = reinterpret_cast<uint64_t *>(at + 16 + 2 * kItemWords * 4);
    full = asked + 1;
    empty = full + 2;
    want = empty + 2;
  }
  __device__ __forceinline__ void init(int readers) const {  // one thread
    mbar_init(asked, 1);
    mbar_init(want, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], readers);
    }
  }
  // asks for another CTA's index (one lane; not again after an empty answer)
  __device__ __forceinline__ void ask() const {
    mbar_arrive_expect_tx(asked, 16);
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128"
        " [%0], [%1];" ::"r"(smem_addr(answer)),
        "r"(smem_addr(asked))
        : "memory");
  }
  // the index, or -1 (every lane, after `asked`)
  __device__ __forceinline__ int answered() const {
    uint32_t got, x = 0;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
        "ld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %1, 1, 0, p;\n\t"
        "mov.u32 %0, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n\t}"
        : "=r"(x), "=r"(got)
        : "r"(smem_addr(answer))
        : "memory");
    fence_proxy_async_smem();  // read before the next answer is written
    return got ? (int)x : -1;
  }
};

// The asking warp's side.  find(index, words) fills in an item and says whether
// it holds work; words[0] < 0 marks the end.
template <class Find> struct ItemSource {
  const ItemRing &ring;
  const Waits &wait;
  Find find;
  int lane;
  int index, count = 0, asks = 0;  // index: the CTA's own, -1 after the end
  __device__ __forceinline__ ItemSource(const ItemRing &r, const Waits &w, Find f, int first,
                                        int l)
      : ring(r), wait(w), find(f), lane(l), index(first) {}
  // Publishes the next item (or the end) into its slot; false when a wait gave
  // up.  words: the item, in every lane.
  __device__ __forceinline__ bool publish(int (&words)[kItemWords]) {
    bool work = false;
    if (count == 0) {
      work = index >= 0 && find(index, words);
    } else if (!wait.all_item(ring.want, (count - 1) & 1)) {
      return false;
    }
    while (index >= 0 && !work) {
      if (elect_one()) ring.ask();
      __syncwarp();
      if (!wait.all(ring.asked, asks & 1)) {  // the answer still comes: not after the CTA left
        mbar_wait_bounded(ring.asked, asks & 1, wait.limit, wait.status);
        return false;
      }
      ++asks;
      index = uniform(ring.answered());
      __syncwarp();
      if (index >= 0) work = find(index, words);
    }
    if (!work) words[0] = -1;
    const int s = count & 1;
    if (!wait.all(&ring.empty[s], ((count >> 1) & 1) ^ 1)) return false;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < kItemWords; ++i) ring.slots[s * kItemWords + i] = words[i];
      mbar_arrive(&ring.full[s]);
    }
    __syncwarp();
    ++count;
    return true;
  }
};

// The reading side (a whole warp): item number `count`; false at the end or when
// a wait gave up.  LOADS: this is the loading warp, whose request starts the
// search for every item but the first.
template <bool LOADS>
__device__ __forceinline__ bool next_item(const ItemRing &ring, const Waits &wait, int &count,
                                          int lane, int (&words)[kItemWords]) {
  const int s = count & 1;
  if (LOADS && count > 0 && lane == 0) mbar_arrive(ring.want);
  if (!wait.all_item(&ring.full[s], (count >> 1) & 1)) return false;
#pragma unroll
  for (int i = 0; i < kItemWords; ++i) {
    words[i] = uniform(ring.slots[s * kItemWords + i]);
  }
  __syncwarp();
  if (lane == 0) mbar_arrive(&ring.empty[s]);
  ++count;
  return words[0] >= 0;
}

// The copies of this thread's stores out of shared memory have been read from
// there, or have arrived.
__device__ __forceinline__ void bulk_stores_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_stores_done() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// 32 rows x W columns (64 or 32) of bf16 to global memory by a warp that holds a
// row per lane (pk: its W / 2 words), through a staging tile of 64 W bytes
// (16-byte pieces swizzled by the row as the tensor map has it: 128-byte rows by
// 8, aligned to 1024; 64-byte rows by 4 in pairs, aligned to 512).  A whole group
// of rows leaves by one tile store, which the warp does not wait for; of a group
// that a sequence ends in, W / 8 lanes store a row's bytes together (straight from
// the lanes, every 16-byte piece would be a transaction of its own).  Rows at or
// past `rows`, columns at or past n: not stored.  map: the output in boxes of 32
// tokens x one head x W columns; (col, head, row) in it is `base`.
template <int W>
__device__ __forceinline__ void store_rows(unsigned char *stage, const uint32_t (&pk)[W / 2],
                                           bf16 *base, int64_t ld, int rows, int n, int lane,
                                           const CUtensorMap *map, int col, int head, int row) {
  constexpr int kPieces = W / 8;  // per row
  uint4 *st = reinterpret_cast<uint4 *>(stage);
  auto swizzle = [](int r) { return W == 64 ? r & 7 : (r >> 1) & 3; };
  bulk_stores_read();  // the last tile has left the staging
  __syncwarp();
#pragma unroll
  for (int c = 0; c < kPieces; ++c)
    st[lane * kPieces + (c ^ swizzle(lane))] =
        make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
  if (rows >= 32) {
    fence_proxy_async_smem();
    __syncwarp();
    if (n > 0 && elect_one()) {
      asm volatile(
          "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
          ::"l"(reinterpret_cast<uint64_t>(map)),
          "r"(col), "r"(head), "r"(row), "r"(smem_addr(stage))
          : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
    __syncwarp();
    return;
  }
  __syncwarp();
  const int c = lane % kPieces;
  if (8 * c < n) {
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int r = 32 / kPieces * k + lane / kPieces;
      if (r < rows)
        *reinterpret_cast<uint4 *>(base + (int64_t)r * ld + 8 * c) =
            st[r * kPieces + (c ^ swizzle(r))];
    }
  }
  __syncwarp();
}

// Sequences by length, the longest first, for batches of 2 to kSortMax: with
// items handed out in this order the long ones do not come last.  Measured
// against the order of the slots: forward 32,768 tokens of 16 to 8,192 x 32/8 x
// 128 1,070 against 1,108 us, 16,384 tokens of 16 to 2,048 x 14/2 x 64 50 against
// 53, backward of the latter 165 against 171.  Larger batches keep the order of
// the slots, which needs no table.  Every CTA makes the same table, from one
// look at cu.
constexpr int kSortMax = 128;

struct SeqOrder {
  int *base;       // [kSortMax]: units of the sequences before rank r
  uint8_t *order;  // [kSortMax]: the sequence of rank r
  int total;       // units of all
  static constexpr uint32_t kBytes = kSortMax * 5;

  __device__ __forceinline__ explicit SeqOrder(unsigned char *at)
      : base(reinterpret_cast<int *>(at)), order(at + kSortMax * 4), total(0) {}

  // All threads of the CTA (at least kSortMax).  tmp: kSortMax + 1 ints of shared
  // memory (16-byte aligned) that tiles are loaded into later.  units(len): work
  // units of a sequence.
  template <class Units>
  __device__ __forceinline__ void make(const AttnArgs &a, int *tmp, Units units) {
    const int b = threadIdx.x;
    int len = -1;
    if (b < a.B) {
      const int c0 = min(max(__ldg(a.cu + b), 0), (int)a.T);
      len = min(max(__ldg(a.cu + b + 1), c0), (int)a.T) - c0;
    }
    if (b < kSortMax) tmp[b] = len;
    __syncthreads();
    if (b < a.B) {
      int rank = 0;
#pragma unroll 8
      for (int c = 0; c < a.B; c += 4) {
        const int4 v = reinterpret_cast<const int4 *>(tmp)[c >> 2];
        rank += v.x > len || (v.x == len && c < b);
        rank += v.y > len || (v.y == len && c + 1 < b);
        rank += v.z > len || (v.z == len && c + 2 < b);
        rank += v.w > len || (v.w == len && c + 3 < b);
      }
      order[rank] = (uint8_t)b;
    }
    __syncthreads();
    if (threadIdx.x < 32) {  // running sum of the units, four ranks per lane
      const int l = threadIdx.x;
      int n[4], s = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * l + i;
        n[i] = r < a.B ? units(tmp[order[r]]) : 0;
        s += n[i];
      }
      int upto = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (l >= o) upto += v;
      }
      int at = upto - s;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        base[4 * l + i] = at;
        at += n[i];
      }
      if (l == 31) tmp[kSortMax] = upto;
    }
    __syncthreads();
    total = tmp[kSortMax];
    fence_proxy_async_smem();  // tmp is written by tile loads next
    __syncthreads();
  }
  // The rank that unit u (< total) belongs to.
  __device__ __forceinline__ int rank_of(int u, int B) const {
    int lo = 0, hi = B - 1;  // the last r with base[r] <= u
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (base[mid] <= u)
        lo = mid;
      else
        hi = mid - 1;
    }
    return lo;
  }
};

// Zeroes rows [from, 128) of a staged tile (whole warp): rows behind a
// sequence's end hold another sequence's values, whose infinities would turn a
// zero probability's product into NaN.
template <int DP>
__device__ __forceinline__ void zero_rows(unsigned char *tile, int from, int lane) {
#pragma unroll
  for (int j = 0; j < DP / 64; ++j) {
    uint4 *p = reinterpret_cast<uint4 *>(tile + j * kBoxBytes);
    for (int i = from * 8 + lane; i < kTile * 8; i += 32) p[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

}  // namespace attn
}  // namespace ftk
