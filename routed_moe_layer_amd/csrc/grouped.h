// Device helpers of the products grouped by expert (grouped.hip).
#pragma once

#include "common.h"
#include "kernels.h"

namespace rmoe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

template <int V>
struct IntC { static constexpr int value = V; };

// Operand types by their moe_quant_t value: 0 BF16, 1 int8, 3 E4M3.
template <int Q> struct AccOf { typedef f32x4 type; };
template <> struct AccOf<1> { typedef i32x4 type; };

// acc += A * B over one 128-byte chunk of K (two 16-byte fragments per lane and operand).
// Any order of K inside the chunk gives the same sum as long as both operands use it.
template <int Q>
__device__ __forceinline__ typename AccOf<Q>::type mma_chunk(u32x4 a0, u32x4 a1, u32x4 b0,
                                                             u32x4 b1,
                                                             typename AccOf<Q>::type acc) {
  if constexpr (Q == 0) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a0),
                                                  __builtin_bit_cast(bf16x8, b0), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a1),
                                                  __builtin_bit_cast(bf16x8, b1), acc, 0, 0, 0);
  } else if constexpr (Q == 1) {
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a0),
                                                __builtin_bit_cast(i32x4, b0), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a1),
                                                __builtin_bit_cast(i32x4, b1), acc, 0, 0, 0);
  } else {
    i32x8 x, y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = static_cast<int>(a0[i]); x[4 + i] = static_cast<int>(a1[i]);
      y[i] = static_cast<int>(b0[i]); y[4 + i] = static_cast<int>(b1[i]);
    }
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc, 0, 0, 0, 0x7F7F7F7F, 0,
                                                           0x7F7F7F7F);   // scales 2^0
  }
  return acc;
}

// Rows of expert e, kept inside [0, R] whatever the prefix sums hold.
__device__ __forceinline__ int2 expert_rows(const GroupedArgs& a, int e) {
  const int lo = e > 0 ? min(max(a.cumsum[e - 1], 0), a.R) : 0;
  const int hi = min(max(a.cumsum[e], lo), a.R);
  return make_int2(lo, hi);
}

// s_tile[e] = number of tiles (of up to BM rows) of the experts before e, s_tile[E] the
// total.  Every thread of the workgroup calls this; it ends with a barrier.
template <int BM, int NW>
__device__ __forceinline__ void scan_tiles(const GroupedArgs& a, int32_t* s_tile) {
  __shared__ int32_t s_wave[NW];
  constexpr int kThreads = NW * 64;
  const int per = (a.E + kThreads - 1) / kThreads;
  const int lo = min(static_cast<int>(threadIdx.x) * per, a.E), hi = min(lo + per, a.E);
  int sum = 0;
  for (int e = lo; e < hi; ++e) {
    const int2 r = expert_rows(a, e);
    const int n = (r.y - r.x + BM - 1) / BM;
    s_tile[e] = n;
    sum += n;
  }
  int inc = sum;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int v = __shfl_up(inc, off);
    if (lane >= off) inc += v;
  }
  if (lane == 63) s_wave[wave] = inc;
  __syncthreads();
  int before = inc - sum;
  for (int i = 0; i < wave; ++i) before += s_wave[i];
  for (int e = lo; e < hi; ++e) {
    const int n = s_tile[e];
    s_tile[e] = before;
    before += n;
  }
  if (threadIdx.x == kThreads - 1) s_tile[a.E] = before;
  __syncthreads();
}

struct TileRows {
  int expert, row0, nrows;
};
// The tile's expert (the last one that starts at or before it) and rows; 0 <= tile < s_tile[E].
template <int BM>
__device__ __forceinline__ TileRows find_tile(const GroupedArgs& a, const int32_t* s_tile, int tile) {
  int lo = 0, hi = a.E;                  // s_tile[lo] <= tile < s_tile[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s_tile[mid] <= tile) lo = mid; else hi = mid;
  }
  const int e = __builtin_amdgcn_readfirstlane(lo);
  const int2 r = expert_rows(a, e);
  const int row0 = r.x + (tile - s_tile[e]) * BM;
  return TileRows{e, row0, min(BM, r.y - row0)};
}

// The same with an expert's rows dealt evenly to its tiles in multiples of 16 (so none is
// nearly empty while others are full); the last tiles of an expert may hold no row.
template <int BM>
__device__ __forceinline__ TileRows find_tile_even(const GroupedArgs& a, const int32_t* s_tile,
                                                   int tile) {
  TileRows t = find_tile<BM>(a, s_tile, tile);
  const int2 r = expert_rows(a, t.expert);
  const int cnt = r.y - r.x, nt = (cnt + BM - 1) / BM;
  const int per = ((cnt + nt - 1) / nt + 15) / 16 * 16;
  t.row0 = r.x + (tile - s_tile[t.expert]) * per;
  t.nrows = min(per, r.y - t.row0);
  return t;
}

// Row of x that sorted row i reads, or -1 (zeros) when the index points outside x.
__device__ __forceinline__ int64_t source_row(const GroupedArgs& a, int i) {
  int s = i;
  if (a.row_idx) {
    s = a.row_idx[i];
    if (s < 0) return -1;
    if (a.row_div > 1) s = static_cast<int>(static_cast<uint32_t>(s) / static_cast<uint32_t>(a.row_div));
  }
  return s < a.x_rows ? s : -1;
}

// tanh(v): an odd polynomial for |v| < 1/4 (next Taylor term below 2^-26 of the value),
// where 1 - exp(-2|v|) would cancel; else (1 - e) / (1 + e), e = exp(-2|v|).
__device__ __forceinline__ float tanh_f32(float v) {
  const float u = fabsf(v), z = v * v;
  const float e = __builtin_amdgcn_exp2f(-2.8853900817779268f * u);
  const float far = (1.0f - e) * __builtin_amdgcn_rcpf(1.0f + e);
  float p = __builtin_fmaf(z, 62.0f / 2835.0f, -17.0f / 315.0f);
  p = __builtin_fmaf(z, p, 2.0f / 15.0f);
  p = __builtin_fmaf(z, p, -1.0f / 3.0f);
  const float near = __builtin_fmaf(u * z, p, u);
  return copysignf(u < 0.25f ? near : far, v);
}

// SiTU(g, u) = (beta tanh(g / beta) sigmoid(g)) * (lambda tanh(u / lambda)).
__device__ __forceinline__ float situ_f32(float g, float u, float beta, float inv_beta, float lam,
                                          float inv_lam) {
  const float sig = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * g));
  return (beta * tanh_f32(g * inv_beta) * sig) * (lam * tanh_f32(u * inv_lam));
}

// One lane's four output columns n0 .. n0 + 3 of one token row: scales, activation, one
// rounding to BF16.  h: the (gate) products, u: the up products of the same columns (SiTU).
template <int Q, bool SITU>
__device__ __forceinline__ void store4(const GroupedArgs& a, int e, int n0,
                                       typename AccOf<Q>::type h, typename AccOf<Q>::type u,
                                       float xs, uint16_t* orow) {
  float v[4];
  float beta = 4.0f, lam = 25.0f;
  if constexpr (SITU) {
    if (a.beta) beta = a.beta[e];
    if (a.lam) lam = a.lam[e];
  }
  const float ib = 1.0f / beta, il = 1.0f / lam;
  const int64_t wrow = static_cast<int64_t>(e) * a.Nw;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = min(n0 + i, a.N - 1);
    float hv = static_cast<float>(h[i]);
    if constexpr (Q != 0) hv = hv * xs * a.w_scale[wrow + n];
    if constexpr (SITU) {
      float uv = static_cast<float>(u[i]);
      if constexpr (Q != 0) uv = uv * xs * a.w_scale[wrow + a.N + n];
      hv = situ_f32(hv, uv, beta, ib, lam, il);
    }
    v[i] = hv;
  }
  if (n0 + 4 <= a.N && a.N % 4 == 0) {
    uint2 o;
    o.x = pack_bf16x2(v[0], v[1]);
    o.y = pack_bf16x2(v[2], v[3]);
    *reinterpret_cast<uint2*>(orow + n0) = o;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n0 + i < a.N) orow[n0 + i] = f32_to_bf16(v[i]);
  }
}

}  // namespace rmoe
