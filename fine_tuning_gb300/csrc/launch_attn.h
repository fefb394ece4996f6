// Launchers of the attention kernels and of the rotation by positions on several
// axes, called by ftk_api.cu.  (Apart from launch.h, which every kernel of the
// per-token path is built from: their measured traffic is filed under a hash of
// their sources and shared headers.)
#pragma once

#include "launch.h"

namespace ftk {

// Rotation of q, k (into oq, ok; may be q, k) by positions on several axes
// (qk_mrope.cu): frequency i turns by pos[axis_of[i] * ld_pos + t].
struct QkMropeArgs {
  const void *q;
  int64_t ld_q;
  const void *k;
  int64_t ld_k;
  void *oq;
  int64_t ld_oq;
  void *ok;
  int64_t ld_ok;
  const int32_t *pos;  // [axes, T], row stride ld_pos
  int64_t ld_pos;
  const int32_t *axis_of;  // HOST [D/2]
  int64_t T;
  int32_t Hq, Hkv, D;
  double theta;
  const double *inv_freq;  // HOST [D/2], nullable
  bool backward;
};
cudaError_t launch_qk_mrope(DType dt, bool vec, const QkMropeArgs &a, const DeviceInfo &dev,
                            cudaStream_t s);

// Attention over packed sequences (attn_*.cu).  Forward: q, k, v in, o and
// lse ([Hq, T], nullable) out.  Backward: do_, q, k, v, o, lse in, dq, dk, dv
// out, delta ([Hq, T] fp32, workspace) in between.
struct AttnArgs {
  const void *q;
  int64_t ld_q;
  const void *k;
  int64_t ld_k;
  const void *v;
  int64_t ld_v;
  void *o;
  int64_t ld_o;
  float *lse;
  const int32_t *cu;
  int32_t B;
  int64_t T;
  int32_t Hq, Hkv, D;
  float scale;
  int32_t causal;
  const uint32_t *skip;  // DEVICE word: non-zero leaves every output untouched
  const void *do_;
  int64_t ld_do;
  void *dq;
  int64_t ld_dq;
  void *dk;
  int64_t ld_dk;
  void *dv;
  int64_t ld_dv;
  float *delta;
};
constexpr int kAttnMaxD = 256;
constexpr float kAttnMaxScale = 0x1p127f;  // log2(e) times it is finite
constexpr int64_t kAttnMaxT = (int64_t(1) << 31) - 1024;
constexpr int kAttnMinTile = 32;  // rows of the smallest tile any attention kernel uses
cudaError_t launch_attn_fwd_generic(DType dt, const AttnArgs &a, const DeviceInfo &dev,
                                    cudaStream_t s);
cudaError_t launch_attn_bwd_generic(DType dt, const AttnArgs &a, const DeviceInfo &dev,
                                    cudaStream_t s);
// bf16, D % 8 == 0, D <= 128, 16-byte aligned tensors, row strides % 8 == 0.
cudaError_t launch_attn_fwd_tc(const AttnArgs &a, const DeviceInfo &dev, cudaStream_t s);
// bytes from AttnArgs::delta on that launch_attn_bwd_tc uses
size_t attn_bwd_tc_workspace_bytes(int64_t T, int32_t Hq, int32_t Hkv, int32_t D);
cudaError_t launch_attn_bwd_tc(const AttnArgs &a, const DeviceInfo &dev, cudaStream_t s);

}  // namespace ftk
