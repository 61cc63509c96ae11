// Microscaled FP4 rows (MXFP4): blocks of 32 values, each with one E8M0 scale byte b (2^(b-127),
// 255: NaN) and E2M1 codes, two per byte, element 2i in the low nibble of byte i.
//   quantize:    b = max(floor(log2 max|v|) - 2 + 127, 0),  code = E2M1(v * 2^(127-b))
//   dequantize:  v = BF16(E2M1(code) * 2^(b-127))
// The scale comes from the exponent field of the largest magnitude alone; quotients by a power
// of two are exact, so the code's rounding (nearest, ties to even, saturating at 6) is the only
// one.  A block with a NaN or an infinity gets b = 255 and codes 0.
//
// A row's scales take whole dwords, so sixteen lanes own one: 128 values, 8 per lane, four lanes
// per block.  Where K is a multiple of 128 these units lie next to each other over the borders of
// rows and need no division.
#include "common.h"
#include "kernels.h"

namespace rmoe {

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

constexpr int kMxThreads = 256;

template <int CTRL>
__device__ __forceinline__ uint32_t dpp32(uint32_t x) {
  return static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(static_cast<int>(x), static_cast<int>(x), CTRL, 0xF, 0xF, false));
}

// The largest of the eight BF16 magnitudes (15 bits; NaNs above infinity above the finite ones)
// over the lane's quad.
__device__ __forceinline__ uint32_t quad_max_magnitude(u32x4 v) {
  u16x2 m = __builtin_bit_cast(u16x2, v[0] & 0x7FFF7FFFu);
#pragma unroll
  for (int i = 1; i < 4; ++i)
    m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[i] & 0x7FFF7FFFu));
  uint32_t x = max(static_cast<uint32_t>(m[0]), static_cast<uint32_t>(m[1]));
  x = max(x, dpp32<0xB1>(x));                          // quad_perm [1,0,3,2]
  return max(x, dpp32<0x4E>(x));                       // quad_perm [2,3,0,1]
}

// Eight BF16 values over 2^(b-127) to E2M1: the conversion divides by its scale's power of two.
__device__ __forceinline__ uint32_t mx_codes8(u32x4 v, uint32_t b) {
  const float s = __uint_as_float(b << 23);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, as_bf16x2(v[0]), s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, as_bf16x2(v[1]), s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, as_bf16x2(v[2]), s, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, as_bf16x2(v[3]), s, 3);
  return b == 255u ? 0u : w;
}

// Where unit u and this lane's eight values of it lie: their index among the rows' values, and
// whether the row has them.
template <bool WHOLE>
__device__ __forceinline__ bool mx_unit(const MxRowsArgs& a, uint32_t u, int l16, int64_t* at) {
  if constexpr (WHOLE) {
    *at = static_cast<int64_t>(u) * 128 + 8 * l16;
    return true;
  } else {
    const uint32_t row = u / a.units;
    const int k = static_cast<int>(u - row * a.units) * 128 + 8 * l16;
    *at = static_cast<int64_t>(row) * a.K + k;
    return k < a.K;
  }
}

template <bool WHOLE>
__global__ __launch_bounds__(kMxThreads) void quantize_mxfp4_kernel(MxRowsArgs a) {
  const uint32_t step = gridDim.x * (kMxThreads / 16);
  const int l16 = threadIdx.x & 15;
  for (uint32_t u = (blockIdx.x * kMxThreads + threadIdx.x) / 16; u < a.total; u += step) {
    int64_t at;
    const bool in = mx_unit<WHOLE>(a, u, l16, &at);
    u32x4 v = {0u, 0u, 0u, 0u};
    if (in) v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(a.src + at));
    const uint32_t e = quad_max_magnitude(v) >> 7;
    const uint32_t b = e == 255u ? 255u : e > 2u ? e - 2u : 0u;
    if (in) *reinterpret_cast<uint32_t*>(a.codes + at / 2) = mx_codes8(v, b);
    uint32_t w = b << (8 * (l16 >> 2));
    w |= dpp32<0x124>(w);                              // row_ror:4
    w |= dpp32<0x128>(w);                              // row_ror:8
    if (l16 == 0) reinterpret_cast<uint32_t*>(a.scales)[u] = w;
  }
}

template <bool WHOLE>
__global__ __launch_bounds__(kMxThreads) void dequantize_mxfp4_kernel(MxRowsArgs a) {
  const uint32_t step = gridDim.x * (kMxThreads / 16);
  const int l16 = threadIdx.x & 15;
  for (uint32_t u = (blockIdx.x * kMxThreads + threadIdx.x) / 16; u < a.total; u += step) {
    int64_t at;
    if (!mx_unit<WHOLE>(a, u, l16, &at)) continue;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(a.codes + at / 2);
    const uint32_t b = reinterpret_cast<const uint32_t*>(a.scales)[u] >> (8 * (l16 >> 2)) & 255u;
    const float s = __uint_as_float(b << 23);          // 0: the conversion takes it for 2^-127
    u32x4 o;
    o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
    o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
    o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
    o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
    if (b == 255u) o = u32x4{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
    *reinterpret_cast<u32x4*>(a.out + at) = o;
  }
}

static unsigned mx_grid(const MxRowsArgs& a) {
  const uint32_t per = kMxThreads / 16, blocks = (a.total + per - 1) / per;
  return blocks < 16u * a.cus ? blocks : 16u * a.cus;
}

hipError_t launch_quantize_mxfp4(const MxRowsArgs& a, hipStream_t stream) {
  const dim3 grid(mx_grid(a)), block(kMxThreads);
  if (a.K % 128 == 0) quantize_mxfp4_kernel<true><<<grid, block, 0, stream>>>(a);
  else quantize_mxfp4_kernel<false><<<grid, block, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_dequantize_mxfp4(const MxRowsArgs& a, hipStream_t stream) {
  const dim3 grid(mx_grid(a)), block(kMxThreads);
  if (a.K % 128 == 0) dequantize_mxfp4_kernel<true><<<grid, block, 0, stream>>>(a);
  else dequantize_mxfp4_kernel<false><<<grid, block, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace rmoe
