// Weighted sum of expert rows back into tokens:
//   out[t] = BF16(add[t] + sum_j w[t, j] * rows[idx[t*k + j]])
// in j order in fp32 (add last, as one more term), rows whose index is negative or past the
// last row left out.  One thread per 8 columns of a token; the index and weight loads are
// uniform over the workgroup.
//
// Bound by the rows' bytes, each read once: 16384 tokens x 16 rows of 3584 take 0.40 ms, 5.0
// TB/s (a large copy on the same card 4.96 TB/s, a large read 5.99).
#include "common.h"
#include "kernels.h"

namespace rmoe {

// BATCH: rows of a token in flight per thread.  NT: rows are read past the caches.
template <int BATCH, bool NT>
__global__ __launch_bounds__(512) void combine_kernel(CombineArgs a) {
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
  for (int j0 = 0; j0 < a.k; j0 += BATCH) {
    u32x4 v[BATCH];
    int64_t r[BATCH];
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      r[j] = j0 + j < a.k ? idx[j0 + j] : -1;
      if (r[j] >= a.R) r[j] = -1;
      if (r[j] >= 0) {
        const u32x4* src = reinterpret_cast<const u32x4*>(a.rows + r[j] * a.H) + p;
        v[j] = NT ? __builtin_nontemporal_load(src) : *src;
      }
    }
#pragma unroll
    for (int j = 0; j < BATCH; ++j)
      if (r[j] >= 0) add8(v[j], bf16_to_f32(wt[j0 + j]));
  }
  if (a.add) add8(reinterpret_cast<const u32x4*>(a.add + t * a.H)[p], 1.0f);
  u32x4 o;
#pragma unroll
  for (int q = 0; q < 4; ++q) o[q] = pack_bf16x2(acc[2 * q], acc[2 * q + 1]);
  reinterpret_cast<u32x4*>(a.out + t * a.H)[p] = o;
}

// With few wavefronts (below 16 per CU) a token's row is spread over workgroups of one and all
// its rows are read at once, through the caches that the products left them in: 256 tokens x
// 16 rows of 3584 8.9 us, 12.1 us the other way.  With many, a workgroup covers as much of a
// row as it can, reads four rows at a time and past the caches: 16384 tokens 399 us, 410 us
// with workgroups of one and eight rows, 438 us with sixteen.
hipError_t launch_combine(const CombineArgs& a, hipStream_t stream) {
  const int waves = (a.H / 8 + 63) / 64;               // per token
  const bool few = a.T * waves < 16 * static_cast<int64_t>(a.cus);
  const int blocks = few ? waves : (waves + 7) / 8, threads = (waves + blocks - 1) / blocks * 64;
  const dim3 grid(static_cast<unsigned>(a.T), static_cast<unsigned>(blocks));
  if (few) combine_kernel<16, false><<<grid, dim3(threads), 0, stream>>>(a);
  else combine_kernel<4, true><<<grid, dim3(threads), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace rmoe
