// Root-mean-square norm of BF16 rows with the residual's addition, and its output as BF16
// rows and as 8-bit codes with one scale per row:
//   h = x + res;  y = h * (1 / sqrt(mean(h^2) + eps)) * w;
//   scale = max|y| / M, code = RN(y / scale) with M = 127 (int8) or 448 (E4M3).
// h, the mean and y are fp32 throughout: h is rounded to BF16 only where it is stored (the
// residual stream), y only where it is stored; the codes come from the unrounded y.  A row
// whose squares would leave fp32's range is multiplied by a power of two first, which cancels
// in y.
//
// Bound by the bytes: each input is read once and held in registers over the two reductions.
// 16384 rows of 3584 with the residual, its sum, BF16 and E4M3 rows (529 MB) take 92 us, 5.8
// TB/s (107 to 114 us after twenty calls in a row; a large copy on the same card 4.96 TB/s, a
// large read 5.99).
#include "common.h"
#include "kernels.h"

namespace rmoe {

template <class F, class T>
__device__ __forceinline__ T wave_reduce(T v, F f) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = f(v, __shfl_xor(v, off));
  return v;
}

constexpr int kNormMaxWaves = 16;

// Sums of squares outside [2^-96, 2^100] are taken again of the scaled row.  Below, a square
// (off by up to 2^-150 where it is subnormal) may have lost bits that count, unless eps of at
// least 2^-80 hides them; above, the sum of a larger row could be infinite.
constexpr float kSumLow = 0x1p-96f, kSumHigh = 0x1p100f, kEpsLow = 0x1p-80f;
// 2^-exponent of the row's largest |h| (bits), 1 for a row of zeros or one that holds an
// infinity.  At most 2^100: with eps < 2^-80 its square times eps stays finite, and the
// smallest BF16 values, 2^-133, still have squares of 2^-66.
__device__ __forceinline__ float row_scale(uint32_t bits) {
  if (bits == 0u || bits >= 0x7F800000u) return 1.0f;
  const int e = min(max(127 - static_cast<int>(bits >> 23), -126), 100);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// One row per workgroup.  A thread holds C pieces of 8 values: piece p = thread + i * threads.
// (A row per wavefront with more pieces each was slower: 16384 rows of 3584 108 us, one row
// 6.6 us against 3.7.)
template <int C>
__global__ __launch_bounds__(kNormMaxWaves * 64) void rmsnorm_kernel(NormArgs a) {
  __shared__ float s_sum[kNormMaxWaves];
  __shared__ uint32_t s_max[kNormMaxWaves];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int per_row = static_cast<int>(blockDim.x), at = static_cast<int>(threadIdx.x);
  const int64_t t = blockIdx.x;
  const int nvec = a.H / 8;
  const u32x4* xr = reinterpret_cast<const u32x4*>(a.x + t * a.H);
  const u32x4* rr = a.res ? reinterpret_cast<const u32x4*>(a.res + t * a.H) : nullptr;
  const u32x4* wr = reinterpret_cast<const u32x4*>(a.weight);
  u32x4 xv[C], rv[C];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int p = at + i * per_row;
    xv[i] = u32x4{0, 0, 0, 0};
    rv[i] = u32x4{0, 0, 0, 0};
    if (p < nvec) {
      xv[i] = __builtin_nontemporal_load(xr + p);
      if (rr) rv[i] = __builtin_nontemporal_load(rr + p);
    }
  }
  float h[C][8];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < C; ++i) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      h[i][2 * q] = __uint_as_float(xv[i][q] << 16);
      h[i][2 * q + 1] = __uint_as_float(xv[i][q] & 0xFFFF0000u);
      if (rr) {
        h[i][2 * q] += __uint_as_float(rv[i][q] << 16);
        h[i][2 * q + 1] += __uint_as_float(rv[i][q] & 0xFFFF0000u);
      }
      ss = __builtin_fmaf(h[i][2 * q], h[i][2 * q], ss);
      ss = __builtin_fmaf(h[i][2 * q + 1], h[i][2 * q + 1], ss);
    }
    const int p = at + i * per_row;
    if (a.res_out && p < nvec) {
      u32x4 o;
#pragma unroll
      for (int q = 0; q < 4; ++q) o[q] = pack_bf16x2(h[i][2 * q], h[i][2 * q + 1]);
      reinterpret_cast<u32x4*>(a.res_out + t * a.H)[p] = o;
    }
  }
  ss = wave_reduce(ss, [](float u, float v) { return u + v; });
  if (lane == 0) s_sum[wave] = ss;
  __syncthreads();
  ss = 0.0f;
  for (int i = 0; i < static_cast<int>(blockDim.x >> 6); ++i) ss += s_sum[i];
  float eps = a.eps;
  if (ss > kSumHigh || (ss < kSumLow && eps < kEpsLow)) {   // uniform; rare
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) big = max(big, __float_as_uint(h[i][e]) & 0x7FFFFFFFu);
    big = wave_reduce(big, [](uint32_t u, uint32_t v) { return max(u, v); });
    if (lane == 0) s_max[wave] = big;
    __syncthreads();
    for (int i = 0; i < static_cast<int>(blockDim.x >> 6); ++i) big = max(big, s_max[i]);
    const float c = row_scale(big);
    ss = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[i][e] *= c;
        ss = __builtin_fmaf(h[i][e], h[i][e], ss);
      }
    eps = eps * c * c;
    ss = wave_reduce(ss, [](float u, float v) { return u + v; });
    if (lane == 0) s_sum[wave] = ss;
    __syncthreads();
    ss = 0.0f;
    for (int i = 0; i < static_cast<int>(blockDim.x >> 6); ++i) ss += s_sum[i];
  }
  const float r = 1.0f / sqrtf(ss / static_cast<float>(a.H) + eps);
  // max|y| as the maximum of the bit patterns: ordered like the values, and a NaN (above
  // every number) stays, so a row that holds one gets a NaN scale instead of losing it.
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int p = at + i * per_row;
    if (p < nvec) {
      const u32x4 w = wr[p];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        h[i][2 * q] = h[i][2 * q] * r * __uint_as_float(w[q] << 16);
        h[i][2 * q + 1] = h[i][2 * q + 1] * r * __uint_as_float(w[q] & 0xFFFF0000u);
        top = max(top, __float_as_uint(h[i][2 * q]) & 0x7FFFFFFFu);
        top = max(top, __float_as_uint(h[i][2 * q + 1]) & 0x7FFFFFFFu);
      }
      if (a.y) {
        u32x4 o;
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = pack_bf16x2(h[i][2 * q], h[i][2 * q + 1]);
        reinterpret_cast<u32x4*>(a.y + t * a.H)[p] = o;
      }
    }
  }
  if (!a.codes) return;
  top = wave_reduce(top, [](uint32_t u, uint32_t v) { return max(u, v); });
  if (lane == 0) s_max[wave] = top;
  __syncthreads();
  for (int i = 0; i < static_cast<int>(blockDim.x >> 6); ++i) top = max(top, s_max[i]);
  const float scale = __uint_as_float(top) / (a.e4m3 ? 448.0f : 127.0f);
  if (at == 0) a.scales[t] = scale;
  // y / scale: the product with the rounded reciprocal and one correction of its residual
  // (the IEEE quotient but for rare last bits; fp32 subnormal scales take the division).
  const bool normal = scale >= 1.1754944e-38f && scale <= 1e37f;
  const float inv = normal ? 1.0f / scale : 0.0f;
  auto quotient = [&](float y) {
    if (!normal) return scale == 0.0f ? 0.0f : y / scale;
    const float q0 = y * inv;
    return __builtin_fmaf(__builtin_fmaf(-scale, q0, y), inv, q0);
  };
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int p = at + i * per_row;
    if (p >= nvec) continue;
    uint2 o;
    uint32_t w[2] = {0u, 0u};
    if (a.e4m3) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float u = fminf(fmaxf(quotient(h[i][2 * q]), -448.0f), 448.0f);
        const float v = fminf(fmaxf(quotient(h[i][2 * q + 1]), -448.0f), 448.0f);
        if (q & 1) w[q >> 1] = __builtin_amdgcn_cvt_pk_fp8_f32(u, v, w[q >> 1], true);
        else w[q >> 1] = __builtin_amdgcn_cvt_pk_fp8_f32(u, v, w[q >> 1], false);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float u = fminf(fmaxf(rintf(quotient(h[i][e])), -127.0f), 127.0f);
        w[e >> 2] |= (static_cast<uint32_t>(static_cast<int32_t>(u)) & 0xFFu) << (8 * (e & 3));
      }
    }
    o.x = w[0];
    o.y = w[1];
    reinterpret_cast<uint2*>(a.codes + t * a.H)[p] = o;
  }
}

hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t stream) {
  const int nvec = a.H / 8;
  // as few pieces per thread as a workgroup's threads allow
  const int threads = nvec <= 1024 ? (nvec + 63) / 64 * 64 : 1024;
  const int per = (nvec + threads - 1) / threads;
  const dim3 grid(static_cast<unsigned>(a.T)), block(threads);
  if (per <= 1) rmsnorm_kernel<1><<<grid, block, 0, stream>>>(a);
  else if (per <= 2) rmsnorm_kernel<2><<<grid, block, 0, stream>>>(a);
  else if (per <= 4) rmsnorm_kernel<4><<<grid, block, 0, stream>>>(a);
  else rmsnorm_kernel<8><<<grid, block, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace rmoe
