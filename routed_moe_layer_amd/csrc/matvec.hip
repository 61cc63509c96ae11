// Products of a few BF16 token rows with an NVFP4 weight matrix (codes and E4M3 block scales
// as moe_quantize_nvfp4 writes them, one fp32 factor alpha):
//   y[t, n] = alpha * sum_b S[n, b] * (sum_{i < 16} E2M1(W[n, 16b + i]) * x[t, 16b + i]).
// An E2M1 value is exact in BF16, so the inner sum is a BF16 dot product accumulated in fp32
// and the block scale multiplies it in fp32: no weight is rounded.
//
// HBM-bound on the 9/16 byte per weight.
#include "common.h"
#include "kernels.h"

namespace rmoe {

// A wavefront computes RW consecutive weight rows for TT tokens; lane l holds block
// 64c + l of every row (16 codes: 8 bytes, one scale byte) and the 16 token values of that
// block, so each load instruction of a row covers 512 contiguous bytes.
template <int RW, int TT>
__global__ __launch_bounds__(256) void matvec_kernel(MatvecArgs a) {
  const int lane = threadIdx.x & 63;
  const int n0 = (static_cast<int>(blockIdx.x) * 4 + static_cast<int>(threadIdx.x >> 6)) * RW;
  const int t0 = static_cast<int>(blockIdx.y) * TT;
  if (n0 >= a.N) return;                                // whole wavefronts; no barrier follows
  const int nb = a.K / 16;
  float acc[RW][TT];
#pragma unroll
  for (int r = 0; r < RW; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[r][t] = 0.0f;
  for (int b = lane; b < nb; b += 64) {
    u32x2 w[RW];
    uint32_t s[RW];
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      const int64_t n = min(n0 + r, a.N - 1);           // rows past the end: the last one again
      w[r] = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(a.codes) + n * nb + b);
      s[r] = a.scales[n * nb + b];
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const int64_t tt = min(t0 + t, a.T - 1);
      const u32x4* xp = reinterpret_cast<const u32x4*>(a.x + tt * a.K) + 2 * b;
      const u32x4 x0 = xp[0], x1 = xp[1];
#pragma unroll
      for (int r = 0; r < RW; ++r)
        acc[r][t] = __builtin_fmaf(e4m3_to_f32(s[r]), e2m1_dot16(w[r], x0, x1), acc[r][t]);
    }
  }
  const float alpha = a.alpha[0];
#pragma unroll
  for (int r = 0; r < RW; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      float v = acc[r][t];
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
      if (lane == 0 && n0 + r < a.N && t0 + t < a.T) {
        const int64_t o = static_cast<int64_t>(t0 + t) * a.N + n0 + r;
        if (a.y_f32) a.y_f32[o] = v * alpha;
        else a.y[o] = f32_to_bf16(v * alpha);
      }
    }
}

hipError_t launch_matvec_nvfp4(const MatvecArgs& a, hipStream_t stream) {
#define RMOE_MATVEC(RW, TT) \
  matvec_kernel<RW, TT><<<dim3((a.N + 4 * RW - 1) / (4 * RW), (a.T + TT - 1) / TT), dim3(256), 0, stream>>>(a)
  if (a.T == 1) RMOE_MATVEC(2, 1);
  else if (a.T == 2) RMOE_MATVEC(2, 2);
  else RMOE_MATVEC(2, 4);
#undef RMOE_MATVEC
  return hipGetLastError();
}

}  // namespace rmoe
