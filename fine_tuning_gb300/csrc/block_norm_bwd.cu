// Backward of the joint of a block's output with the residual stream (block_norm.cuh).
// With xn = x r1, hn = h r2, wg = w_post gate, m the dropout's mask and
// beta = x_scale / (probability of being kept):
//   G    = dh + r2 w dy - k hn,     k = r2 / H sum_j w dy hn
//   dres = res_scale G
//   c    = beta gate_tok sum_j m wg xn G
//   dx   = r1 (beta gate_tok m wg G) - (r1 / H) c xn        (no second term without w_post)
//   dw   = sum_t dy hn,   S = sum_t beta gate_tok m G xn,   dw_post = gate S, dgate = w_post S
//   dgate_tok[t] = c / gate_tok, formed without the division
// Both row sums come from one pass over the row: with q = m wg xn,
//   sum q G = sum q (dh + r2 w dy) - k sum q hn.
// The normalised xn and hn enter the sums, not x and h: no r^3 is formed, which
// overflows for rows near zero.
//
// A CTA's column sums go to its own row of the workspace; a second kernel adds the
// rows in a fixed order and applies gate and w_post.
#include "block_norm.cuh"

namespace ftk {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxBlocksPerSm = 8;

// Rows of any length and alignment: a CTA walks one row at a time, twice.
template <typename T>
__global__ void __launch_bounds__(kThreads) block_norm_bwd_any(const BlockNorm<T> a) {
  __shared__ float red[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const Philox g = philox_of(a.drop);
  float *const sum_w = a.ws + (int64_t)blockIdx.x * 2 * a.H, *const sum_s = sum_w + a.H;
  for_columns(g, 0, 0, a.H, [&](int j, bool) { sum_w[j] = sum_s[j] = 0.f; });
  const float beta = a.x_scale * a.drop.scale;
  for (int64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
    const T *xr = a.x + t * a.ldx, *hr = a.h + t * a.ldh;
    const T *gy = a.dy + t * a.lddy, *gh = a.dh + t * a.lddh;
    const float r1 = a.w_post != nullptr ? a.rstd_post[t] : 1.f, r2 = a.rstd[t];
    const float gt = a.gate_tok != nullptr ? a.gate_tok[t] : 1.f;
    float s_h = 0.f, s_g = 0.f, s_c = 0.f;  // sum w dy hn, sum q (dh + r2 w dy), sum q hn
    for_columns(g, a.drop.thr, t, a.H, [&](int j, bool kept) {
      const float wd = to_float(a.w[j]) * to_float(gy[j]), hn = to_float(hr[j]) * r2;
      const float q = kept ? column_factor(a, j) * (to_float(xr[j]) * r1) : 0.f;
      s_h = fmaf(wd, hn, s_h);
      s_g = fmaf(q, fmaf(r2, wd, to_float(gh[j])), s_g);
      s_c = fmaf(q, hn, s_c);
    });
    s_h = cta_sum(s_h, red, kThreads / 32);
    s_g = cta_sum(s_g, red, kThreads / 32);
    s_c = cta_sum(s_c, red, kThreads / 32);
    const float k = r2 * (s_h * a.inv_h);
    const float c = beta * fmaf(-k, s_c, s_g);
    if (a.dgate_tok != nullptr && threadIdx.x == 0) a.dgate_tok[t] = c;
    const float am = a.w_post != nullptr ? r1 * (gt * c * a.inv_h) : 0.f;
    const float bg = beta * gt;
    for_columns(g, a.drop.thr, t, a.H, [&](int j, bool kept) {
      const float dyf = to_float(gy[j]), hn = to_float(hr[j]) * r2, xn = to_float(xr[j]) * r1;
      const float G = fmaf(-k, hn, fmaf(r2, to_float(a.w[j]) * dyf, to_float(gh[j])));
      const float gm = kept ? bg * G : 0.f;
      sum_w[j] = fmaf(dyf, hn, sum_w[j]);
      sum_s[j] = fmaf(gm, xn, sum_s[j]);
      a.dres[t * a.lddr + j] = from_float<T>(a.res_scale * G);
      a.dx[t * a.lddx + j] = from_float<T>(fmaf(-am, xn, r1 * (gm * column_factor(a, j))));
    });
  }
}

constexpr int kReduceWarps = 32;

// dw[j] = sum_p ws[p][j]; S[j] = sum_p ws[p][H + j], dw_post = gate S, dgate = w_post S.
// A CTA owns 32 columns; its warps take the rows p = warp, warp + 32, ... and their
// sums are added in the warps' order.
template <typename T>
__global__ void __launch_bounds__(32 * kReduceWarps)
block_norm_dw(const float *ws, int P, int H, const T *w_post, const T *gate, float *dw,
              float *dw_post, float *dgate) {
  __shared__ float part[kReduceWarps][33];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j = blockIdx.x * 32 + lane;
  const bool shared = blockIdx.y != 0;  // the column sums that dw_post and dgate share
  float s = 0.f;
  if (j < H)
    for (int p = warp; p < P; p += kReduceWarps)
      s += __ldcg(ws + ((int64_t)p * 2 + (shared ? 1 : 0)) * H + j);
  part[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || j >= H) return;
  float v = 0.f;
#pragma unroll
  for (int i = 0; i < kReduceWarps; ++i) v += part[i][lane];
  if (!shared) {
    dw[j] = v;
    return;
  }
  if (dw_post != nullptr) dw_post[j] = gate != nullptr ? to_float(gate[j]) * v : v;
  if (dgate != nullptr) dgate[j] = w_post != nullptr ? to_float(w_post[j]) * v : v;
}

template <typename T>
cudaError_t reduce(const BlockNormArgs &a, int64_t P, cudaStream_t s) {
  const bool shared = a.dw_post != nullptr || a.dgate != nullptr;
  cudaError_t e = launch_pdl(block_norm_dw<T>,
                             dim3((unsigned)ceil_div(a.H, (int64_t)32), shared ? 2 : 1),
                             dim3(32 * kReduceWarps), 0, s, a.ws, (int)P, (int)a.H,
                             (const T *)a.w_post, (const T *)a.gate, a.dw, a.dw_post, a.dgate);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t bwd_typed(bool, const BlockNormArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  if (a.T == 0) return reduce<T>(a, 0, s);
  const int64_t P = a.T < (int64_t)dev.sms * 4 ? a.T : (int64_t)dev.sms * 4;
  cudaError_t e = launch_pdl(block_norm_bwd_any<T>, dim3((unsigned)P), dim3(kThreads), 0, s,
                             block_norm_params<T>(a));
  return e != cudaSuccess ? e : reduce<T>(a, P, s);
}

}  // namespace

int64_t block_norm_partial_rows(int64_t T, const DeviceInfo &dev) {
  const int64_t cap = (int64_t)dev.sms * kMaxBlocksPerSm;
  return T < cap ? T : cap;
}

cudaError_t launch_block_norm_bwd(DType dt, bool vec, const BlockNormArgs &a,
                                  const DeviceInfo &dev, cudaStream_t s) {
  return dt == DType::F32 ? bwd_typed<float>(vec, a, dev, s) : bwd_typed<bf16>(vec, a, dev, s);
}

}  // namespace ftk
