// Pieces shared by the attention kernels (attn_generic.cu, attn_fwd_tc.cu,
// attn_bwd_tc.cu): how a block finds its sequence and tile from cu_seqlens on
// the device, and the exponential.
//
// Tiles of `tile` rows are numbered without a prefix sum over the sequences:
// sequence b's tiles take the slots from slot_base(b) = floor(cu[b] / tile) + b
// on.  It has ceil(len / tile) <= slot_base(b + 1) - slot_base(b) of them, so
// the ranges never meet, floor(T / tile) + B slots hold every tile, and the
// host needs T and B only.  At most B slots stay empty; a block that gets one
// moves on.
#pragma once

#include "common.cuh"
#include "launch_attn.h"

namespace ftk {

namespace {

// One tile: rows start + row0 .. of the sequence [start, start + len), or
// len = 0 for an empty slot.
struct SeqTile {
  int start, len, row0;
};

// Bounds are clamped into [0, T] with start <= end, so a malformed cu can
// give wrong tiles but no address outside the tensors.
__device__ __forceinline__ SeqTile seq_tile(int slot, const int32_t *cu, int B, int T, int tile) {
  int lo = 1, hi = B;  // first b in [1, B] with slot_base(b) > slot
  while (lo <= hi) {
    const int mid = (lo + hi) >> 1;
    if (max(__ldg(cu + mid), 0) / tile + mid <= slot)
      lo = mid + 1;
    else
      hi = mid - 1;
  }
  const int b = min(lo - 1, B - 1);
  const int c0 = min(max(__ldg(cu + b), 0), T);
  const int c1 = min(max(__ldg(cu + b + 1), c0), T);
  const int64_t row0 = (int64_t)(slot - c0 / tile - b) * tile;
  SeqTile t;
  t.start = c0;
  t.len = (row0 < 0 || row0 >= c1 - c0) ? 0 : c1 - c0;
  t.row0 = (int)(t.len ? row0 : 0);
  return t;
}

// True when the boundary check that ran before this kernel found the batch's
// cu_seqlens malformed; read past L1 after the grid-dependency wait.
__device__ __forceinline__ bool attn_skipped(const uint32_t *skip) {
  return skip != nullptr && __ldcg(skip) != 0u;
}

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

}  // namespace

}  // namespace ftk
