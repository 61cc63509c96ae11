// Weighted sum of expert rows back into tokens:
//   out[t] = BF16(add[t] + sum_j w[t, j] * rows[idx[t*k + j]])
// in j order in fp32 (add last, as one more term), rows whose index is negative or past the
// last row left out.  One thread per 8 columns of a token; the index and weight loads are
// uniform over the workgroup.  HBM-bound: every row is read once.
#include "common.h"
#include "kernels.h"

namespace rmoe {

constexpr int kCombineBatch = 8;          // rows of a token in flight per thread

__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) {
  const int64_t t = blockIdx.x;
  const int nvec = a.H / 8;
  const int p = static_cast<int>(blockIdx.y) * static_cast<int>(blockDim.x) + threadIdx.x;
  if (p >= nvec) return;
  float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  const int32_t* idx = a.idx + t * a.k;
  const uint16_t* wt = a.weights + t * a.k;
  auto add8 = [&](u32x4 v, float w) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      acc[2 * q] = __builtin_fmaf(w, __uint_as_float(v[q] << 16), acc[2 * q]);
      acc[2 * q + 1] = __builtin_fmaf(w, __uint_as_float(v[q] & 0xFFFF0000u), acc[2 * q + 1]);
    }
  };
  for (int j0 = 0; j0 < a.k; j0 += kCombineBatch) {
    u32x4 v[kCombineBatch];
    int64_t r[kCombineBatch];
#pragma unroll
    for (int j = 0; j < kCombineBatch; ++j) {
      r[j] = j0 + j < a.k ? idx[j0 + j] : -1;
      if (r[j] >= a.R) r[j] = -1;
      if (r[j] >= 0)
        v[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(a.rows + r[j] * a.H) + p);
    }
#pragma unroll
    for (int j = 0; j < kCombineBatch; ++j)
      if (r[j] >= 0) add8(v[j], bf16_to_f32(wt[j0 + j]));
  }
  if (a.add) add8(reinterpret_cast<const u32x4*>(a.add + t * a.H)[p], 1.0f);
  u32x4 o;
#pragma unroll
  for (int q = 0; q < 4; ++q) o[q] = pack_bf16x2(acc[2 * q], acc[2 * q + 1]);
  reinterpret_cast<u32x4*>(a.out + t * a.H)[p] = o;
}

hipError_t launch_combine(const CombineArgs& a, hipStream_t stream) {
  const int nvec = a.H / 8;
  const int threads = nvec >= 256 ? 256 : (nvec + 63) / 64 * 64;
  const dim3 grid(static_cast<unsigned>(a.T), static_cast<unsigned>((nvec + threads - 1) / threads));
  combine_kernel<<<grid, dim3(threads), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace rmoe
