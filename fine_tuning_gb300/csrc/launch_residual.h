// Launchers of the residual stream's kernels (embedding, dropout, the joint of a
// block's output with the stream), called by ftk_api.cu.  (Apart from launch.h,
// which every kernel of the per-token path is built from: their measured traffic
// is filed under a hash of their sources and shared headers.)
#pragma once

#include "launch.h"

namespace ftk {

// What a dropout mask is made from (philox.cuh); thr == 0: no dropout.
struct DropArgs {
  uint32_t k0 = 0, k1 = 0;        // the seed's halves
  uint64_t offset = 0;            // further from another's than the run has steps
  const int64_t *step = nullptr;  // DEVICE, nullable: added to offset
  int thr = 0;                    // of 65536: elements whose number is below are dropped
  float scale = 1.f;              // 65536 / (65536 - thr), 0 when everything is dropped
};

// CTAs along the rows for kernels whose threads stay with a packet of columns and walk the
// rows three at a time (`side` rows of a CTA side by side, `parts` CTAs to a row): 64 an
// SM while that leaves a thread two turns, since more CTAs keep the rows in flight closer
// together, and 8 at least.  Measured with 8, 32 and 64 an SM: dropout 65,535 x 4,096 bf16
// 184, 165 and 164 us, lookup of 65,536 x 4,096 126, 117 and 116; dropout 16,384 x 896 (7
// rows a thread with 8) with 8 and 32 10.2 and 12.9.
constexpr int kRowsTurn = 3;
inline int64_t row_grid(int64_t T, int side, int parts, const DeviceInfo &dev) {
  const int64_t all = (T + side - 1) / side, two_turns = all / (2 * kRowsTurn);
  const int64_t least = ((int64_t)dev.sms * 8 + parts - 1) / parts, most = 8 * least;
  const int64_t grid = two_turns < least ? least : two_turns > most ? most : two_turns;
  return grid < all ? grid : all;
}

struct DropoutArgs {
  const void *x;
  int64_t ldx;
  void *y;
  int64_t ldy;
  int64_t T, H;
  DropArgs drop;
};
cudaError_t launch_dropout(DType dt, bool vec, const DropoutArgs &a, const DeviceInfo &dev,
                           cudaStream_t s);

struct EmbedFwdArgs {
  const void *w;
  int64_t ldw, V;
  const int32_t *ids;
  void *x;
  int64_t ldx;
  int64_t T, H;
  float scale;
};
cudaError_t launch_embed_fwd(DType dt, bool vec, const EmbedFwdArgs &a, const DeviceInfo &dev,
                             cudaStream_t s);

struct EmbedBwdArgs {
  const void *dx;
  int64_t lddx;
  const int32_t *ids;
  float *dw;
  int64_t lddw, V;
  int64_t T, H;
  float scale;
  bool accumulate;
  void *ws;
};
// Does not depend on the device: a plan of the sizes alone.
size_t embed_bwd_workspace_bytes(int64_t T, int64_t H, int64_t V);
cudaError_t launch_embed_bwd(DType dt, bool vec, const EmbedBwdArgs &a, cudaStream_t s);

// The joint h = res_scale res + x_scale dropout(gate gate_tok norm(x)), y = norm(h).
struct BlockNormArgs {
  const void *x;
  int64_t ldx;
  const void *res;  // forward
  int64_t ldr;
  const void *w_post, *gate, *w;  // w_post, gate: nullable
  const float *gate_tok;          // nullable
  void *h;  // forward: written; backward: read
  int64_t ldh;
  void *y;
  int64_t ldy;
  float *rstd_post, *rstd;  // forward: nullable, written; backward: read
  int64_t T, H;
  float eps, res_scale, x_scale;
  DropArgs drop;
  // backward
  const void *dy;
  int64_t lddy;
  const void *dh;
  int64_t lddh;
  void *dx;
  int64_t lddx;
  void *dres;
  int64_t lddr;
  float *dw_post, *dgate, *dgate_tok, *dw;
  float *ws;  // [rows][2 H] partial sums of dw and of what dw_post and dgate share
};
cudaError_t launch_block_norm_fwd(DType dt, bool vec, const BlockNormArgs &a,
                                  const DeviceInfo &dev, cudaStream_t s);
// Upper bound on the partial rows of the backward.
int64_t block_norm_partial_rows(int64_t T, const DeviceInfo &dev);
cudaError_t launch_block_norm_bwd(DType dt, bool vec, const BlockNormArgs &a,
                                  const DeviceInfo &dev, cudaStream_t s);

}  // namespace ftk
