// Products of a few BF16 token rows with an NVFP4 weight matrix (codes and E4M3 block scales
// as moe_quantize_nvfp4 writes them, one fp32 factor alpha):
//   y[t, n] = alpha * sum_b S[n, b] * (sum_{i < 16} E2M1(W[n, 16b + i]) * x[t, 16b + i]).
// Bound by the 9/16 byte per weight, and for the smallest by the latency of a launch: one
// token x 16384 x 7168 (66 MB) 14.3 us, 4.6 TB/s; the router's logits, one token x 896 x 3584,
// 3.5 us inside a graph.  With more tokens the token values, which every workgroup reads whole,
// add to it and soon bound it: 16 tokens x 7181 x 7168 (29 MB) 15.0 us, 10.3 without their
// loads; 64 tokens x 16384 x 7168 72 us, with 470 MB of token values for 66 of weights.  Two
// kernels:
// with one or two tokens a wavefront takes whole weight rows, with more the matrix units take
// 16 tokens at a time.
#include <algorithm>

#include "common.h"
#include "kernels.h"

namespace rmoe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------------------------------
// One or two tokens.  A wavefront computes RW consecutive weight rows; lane l holds block
// 64c + l of every row (8 bytes of codes, one scale byte), so a load instruction covers 512
// contiguous bytes of a row, and the codes of the next kDotDepth steps are on their way while
// a step is multiplied.  An E2M1 value is exact in BF16: the inner sum is a BF16 dot product
// accumulated in fp32, multiplied by the block scale in fp32.  The tokens lie in LDS (read once
// per workgroup; every wavefront reading them from the caches moved as many bytes as the
// weights), a block's two 16-byte halves in two planes so that the lanes' reads are
// consecutive.
// ---------------------------------------------------------------------------------------
constexpr int kDotDepth = 4, kDotLdsBytes = 65536;

template <int RW, int TT, int NW, bool LDS>
__global__ __launch_bounds__(NW * 64) void matvec_dot_kernel(MatvecArgs a) {
  extern __shared__ u32x4 s_x[];                       // [TT][2][K / 16]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n0 = (static_cast<int>(blockIdx.x) * NW + wave) * RW;
  const int nb = a.K / 16;
  const u32x4* xg = reinterpret_cast<const u32x4*>(a.x);
  const u32x2* wp[RW];
  const uint8_t* sp[RW];
#pragma unroll
  for (int r = 0; r < RW; ++r) {
    const int64_t n = min(n0 + r, a.N - 1);             // rows past the end: the last one again
    wp[r] = reinterpret_cast<const u32x2*>(a.codes) + n * nb;
    sp[r] = a.scales + n * nb;
  }
  u32x2 w[kDotDepth][RW];
  uint32_t s[kDotDepth][RW];
  auto load = [&](int u, int b) {
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      w[u][r] = u32x2{0, 0};
      s[u][r] = 0;
      if (b < nb) {
        w[u][r] = __builtin_nontemporal_load(wp[r] + b);
        s[u][r] = sp[r][b];
      }
    }
  };
#pragma unroll
  for (int u = 0; u < kDotDepth; ++u) load(u, lane + 64 * u);
  if constexpr (LDS) {
    for (int i = threadIdx.x; i < a.T * nb * 2; i += NW * 64) {
      const int t = i / (2 * nb), h = i - t * 2 * nb;    // half h & 1 of the token's block h / 2
      s_x[(2 * t + (h & 1)) * nb + (h >> 1)] = xg[i];
    }
    __syncthreads();
  }
  if (n0 >= a.N) return;                                // whole wavefronts; no barrier follows
  float acc[RW][TT];
#pragma unroll
  for (int r = 0; r < RW; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[r][t] = 0.0f;
  for (int b0 = lane; b0 - lane < nb; b0 += 64 * kDotDepth) {
#pragma unroll
    for (int u = 0; u < kDotDepth; ++u) {
      const int b = b0 + 64 * u;
      if (b - lane >= nb) break;                        // uniform
      const int bx = min(b, nb - 1);                    // (lanes past the row: zero codes)
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const int tt = min(t, a.T - 1);
        const u32x4 x0 = LDS ? s_x[2 * tt * nb + bx] : xg[(static_cast<int64_t>(tt) * nb + bx) * 2];
        const u32x4 x1 =
            LDS ? s_x[(2 * tt + 1) * nb + bx] : xg[(static_cast<int64_t>(tt) * nb + bx) * 2 + 1];
#pragma unroll
        for (int r = 0; r < RW; ++r) {
          const float d = e2m1_dot16(w[u][r], x0, x1);
          acc[r][t] = __builtin_fmaf(e4m3_to_f32(s[u][r]), b < nb ? d : 0.0f, acc[r][t]);
        }
      }
      load(u, b + 64 * kDotDepth);
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
      if (lane == 0 && n0 + r < a.N && t < a.T) {
        const int64_t o = static_cast<int64_t>(t) * a.N + n0 + r;
        if (a.y_f32) a.y_f32[o] = v * alpha;
        else a.y[o] = f32_to_bf16(v * alpha);
      }
    }
}

// ---------------------------------------------------------------------------------------
// More tokens, 16 TT at a time.  A workgroup takes 16 G weight rows; its wavefronts share K in
// chunks of 128 and add their partial sums through LDS in a fixed order at the end, so few
// rows already fill the chip.  A lane holds 32 consecutive codes of a row (two blocks) and the
// same 32 values of a token: four 16x16x32 BF16 products, K permuted alike in both operands.
// A code times its block scale has at most 6 significant bits: exact in BF16.
// ---------------------------------------------------------------------------------------
// Eight codes (a word) times a block scale, as a BF16 MFMA operand.
__device__ __forceinline__ bf16x8 e2m1_scaled8(uint32_t w, float s) {
  u32x4 r;
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
  const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
  const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
  const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
  r[0] = pack_bf16x2(a[0] * s, a[1] * s);
  r[1] = pack_bf16x2(b[0] * s, b[1] * s);
  r[2] = pack_bf16x2(c[0] * s, c[1] * s);
  r[3] = pack_bf16x2(d[0] * s, d[1] * s);
  return __builtin_bit_cast(bf16x8, r);
}

// PAIRS: K is a multiple of 32, so a lane's two blocks are there or not together and its
// loads are 16 and 2 bytes wide; else each block is looked at by itself.
template <int G, int TT, int NW, bool PAIRS>
__global__ __launch_bounds__(NW * 64) void matvec_mfma_kernel(MatvecArgs a) {
  constexpr int kRows = 16 * G, kStride = kRows + 4;    // floats per token of a partial sum
  __shared__ alignas(16) float red[NW][16 * TT][kStride];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, g = lane >> 4, l16 = lane & 15;
  const int n0 = static_cast<int>(blockIdx.x) * kRows, t0 = static_cast<int>(blockIdx.y) * 16 * TT;
  const int nb = a.K / 16, nc = (a.K + 127) / 128;
  const uint8_t *wp[G], *sp[G];
  const uint16_t* xp[TT];
#pragma unroll
  for (int r = 0; r < G; ++r) {
    const int64_t n = min(n0 + 16 * r + l16, a.N - 1);  // rows past the end: the last one again
    wp[r] = a.codes + n * (a.K / 2) + 16 * g;
    sp[r] = a.scales + n * nb + 2 * g;
  }
#pragma unroll
  for (int t = 0; t < TT; ++t)
    xp[t] = a.x + static_cast<int64_t>(min(t0 + 16 * t + l16, a.T - 1)) * a.K + 32 * g;
  f32x4 acc[G][TT];
#pragma unroll
  for (int r = 0; r < G; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[r][t] = f32x4{0, 0, 0, 0};
  // the next chunk's codes are loaded ahead, and its token values too while they fit
  constexpr int kXDepth = TT <= 2 ? 2 : 1;
  u32x4 w[2][G], xv[kXDepth][TT][4];
  uint32_t s[2][G];
  auto load_w = [&](int u, int c) {
    const int k = 128 * c + 32 * g;
#pragma unroll
    for (int r = 0; r < G; ++r) {
      w[u][r] = u32x4{0, 0, 0, 0};
      s[u][r] = 0;
      if constexpr (PAIRS) {
        if (k < a.K) {
          w[u][r] = *reinterpret_cast<const u32x4*>(wp[r] + 64 * c);
          s[u][r] = *reinterpret_cast<const uint16_t*>(sp[r] + 8 * c);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (k + 16 * h < a.K) {
            const u32x2 v = *reinterpret_cast<const u32x2*>(wp[r] + 64 * c + 8 * h);
            w[u][r][2 * h] = v[0];
            w[u][r][2 * h + 1] = v[1];
            s[u][r] |= static_cast<uint32_t>(sp[r][8 * c + h]) << (8 * h);
          }
      }
    }
  };
  auto load_x = [&](int u, int c) {
    const int k = 128 * c + 32 * g;
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        xv[u][t][q] = u32x4{0, 0, 0, 0};
        if (k + 16 * (q >> 1) < a.K)
          xv[u][t][q] = *reinterpret_cast<const u32x4*>(xp[t] + 128 * c + 8 * q);
      }
  };
  // a wave's chunks are consecutive: two of them share the cache lines of the codes
  const int first = nc * wave / NW, last = nc * (wave + 1) / NW;
  if (first < last) {
    load_w(0, first);
    if constexpr (kXDepth == 2) load_x(0, first);
  }
  for (int c0 = first; c0 < last; c0 += 2) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int c = c0 + u;
      if (c >= last) break;                             // uniform
      constexpr bool kAhead = kXDepth == 2;
      const int v = kAhead ? u : 0;
      if (c + 1 < last) load_w(u ^ 1, c + 1);
      if (!kAhead || c + 1 < last) load_x(kAhead ? u ^ 1 : 0, kAhead ? c + 1 : c);
#pragma unroll
      for (int r = 0; r < G; ++r) {
        const float sf[2] = {e4m3_to_f32(s[u][r]), e4m3_to_f32(s[u][r] >> 8)};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const bf16x8 wq = e2m1_scaled8(w[u][r][q], sf[q >> 1]);
#pragma unroll
          for (int t = 0; t < TT; ++t)
            acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                wq, __builtin_bit_cast(bf16x8, xv[v][t][q]), acc[r][t], 0, 0, 0);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < G; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t)
      *reinterpret_cast<f32x4*>(&red[wave][16 * t + l16][16 * r + 4 * g]) = acc[r][t];
  __syncthreads();
  const float alpha = a.alpha[0];
  for (int i = tid; i < kRows * 16 * TT; i += NW * 64) {
    const int row = i % kRows, t = i / kRows;
    float v = 0.0f;
#pragma unroll
    for (int u = 0; u < NW; ++u) v += red[u][t][row];
    if (n0 + row < a.N && t0 + t < a.T) {
      const int64_t o = static_cast<int64_t>(t0 + t) * a.N + n0 + row;
      if (a.y_f32) a.y_f32[o] = v * alpha;
      else a.y[o] = f32_to_bf16(v * alpha);
    }
  }
}

template <int RW, int TT, int NW>
static hipError_t launch_dot(const MatvecArgs& a, hipStream_t stream) {
  const dim3 grid((a.N + NW * RW - 1) / (NW * RW));
  const size_t lds = static_cast<size_t>(a.T) * a.K * 2;
  if (lds <= kDotLdsBytes)
    matvec_dot_kernel<RW, TT, NW, true><<<grid, dim3(NW * 64), lds, stream>>>(a);
  else
    matvec_dot_kernel<RW, TT, NW, false><<<grid, dim3(NW * 64), 0, stream>>>(a);
  return hipGetLastError();
}

template <int G, int TT, int NW>
static hipError_t launch_mfma(const MatvecArgs& a, hipStream_t stream) {
  const dim3 grid((a.N + 16 * G - 1) / (16 * G), (a.T + 16 * TT - 1) / (16 * TT));
  if (a.K % 32 == 0) matvec_mfma_kernel<G, TT, NW, true><<<grid, dim3(NW * 64), 0, stream>>>(a);
  else matvec_mfma_kernel<G, TT, NW, false><<<grid, dim3(NW * 64), 0, stream>>>(a);
  return hipGetLastError();
}

// One and two tokens: 16 weight rows per workgroup from 24 rows per CU on, 8 below (us with 8
// and 16 rows, one token: N = 896, K = 3584 3.5 and 4.5; N = 2048 3.8 and 4.7; N = 3584 4.8 and
// 5.0; N = 5120 5.8 and 6.5; N = 7168 6.7 and 6.7; N = 16384 11.7 and 10.4; two tokens the same
// way; K = 1792 and 7168 cross between 5120 and 7168 too).  Two tokens stay with the dot
// products (N = 7168 11.8 us against 12.6).
//
// More tokens: 16 G weight rows and 16 TT tokens per workgroup.  A launch takes whole rounds of
// one workgroup per CU, a round the longer the more a workgroup has to do (10, 11, 21, 19 and 30
// for the five shapes: fitted to all the times below); the shape with the smallest product of
// the two is taken.  Measured for N = 256 .. 32768, T = 3 .. 64 and K =
// 1792, 3584 and 7168 (256 CUs, weights from memory), on both sides of each border; us with
// G x TT =              1 x 1   2 x 1   4 x 1   2 x 2   2 x 4
//   16 x 4096  x 7168    13.8    16.9    24.7                     1 round of the smallest
//   16 x 4224  x 7168    23.3    16.8    24.7                     2, 1 and 1 rounds
//   16 x 8192  x 7168    24.9    18.2    25.7
//   16 x 8320  x 7168    34.5    31.1    25.5                     3, 2 and 1
//   16 x 16384 x 3584    24.9    18.5    16.8
//   16 x 16640 x 3584    29.0    24.3    28.7                     5, 3 and 2
//   32 x 2048  x 7168    13.1    16.2    23.7    23.3
//   32 x 4096  x 7168    23.3    16.6    23.9    23.7
//   32 x 4224  x 7168    32.8    28.1    24.2    23.8
//   64 x 2048  x 7168    22.0    16.0    23.3    22.9    35.4
//   64 x 4096  x 7168    41.4    28.6    23.7    23.2    35.8
//   64 x 4224  x 7168    50.0    40.4    43.5    42.1    35.8
//   64 x 16384 x 7168     157     106      88      86      72
// Over all of these the taken shape is at most 12% behind the best (with 3 tokens, whose few
// values make a round of 16 rows shorter than the rule counts), 0.8% on the average; with K of
// 1024 7%, of 160, where a launch is 2 to 6 us and several workgroups run on a CU, 31%.  The sum
// of an output is made in the same order by every shape.
hipError_t launch_matvec_nvfp4(const MatvecArgs& a, hipStream_t stream) {
  if (a.T <= 2) {
    const bool few = a.N < 24 * a.cus;
    if (a.T == 1) return few ? launch_dot<1, 1, 8>(a, stream) : launch_dot<2, 1, 8>(a, stream);
    return few ? launch_dot<1, 2, 8>(a, stream) : launch_dot<2, 2, 8>(a, stream);
  }
  auto cost = [&](int g, int tt, int round) {
    const int groups = ((a.N + 16 * g - 1) / (16 * g)) * ((a.T + 16 * tt - 1) / (16 * tt));
    return (groups + a.cus - 1) / a.cus * round;
  };
  const int c11 = cost(1, 1, 10), c21 = cost(2, 1, 11), c41 = cost(4, 1, 21);
  const int c22 = cost(2, 2, 19), c24 = cost(2, 4, 30);
  const int best = std::min({c11, c21, c41, c22, c24});
  if (best == c11) return launch_mfma<1, 1, 8>(a, stream);
  if (best == c21) return launch_mfma<2, 1, 8>(a, stream);
  if (best == c41) return launch_mfma<4, 1, 8>(a, stream);
  if (best == c22) return launch_mfma<2, 2, 8>(a, stream);
  return launch_mfma<2, 4, 8>(a, stream);
}

}  // namespace rmoe
