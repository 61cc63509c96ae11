// Matrix products grouped by expert with ragged sizes: rows sorted by expert (expert e owns
// rows cumsum[e-1] .. cumsum[e]-1) times that expert's weights [Nw, K],
//   h[i, n] = sum_k x[src(i), k] * W_e[n, k]        (BF16: fp32 accumulation; int8: exact
//             int32; E4M3: fp32), times x_scale[src(i)] * w_scale[e, n] for 8-bit operands,
//   out[i, n] = BF16(h[i, n])   or   BF16(SiTU(h[i, n], h[i, N + n]))  with Nw = 2N.
//
// All three types are handled through the bytes of K: an MFMA operand fragment is 16 bytes
// per lane (lane l: row l % 16, bytes 16 (l / 16) of a 64-byte step), and a K chunk is 128
// bytes = two fragments: two 16x16x32 BF16 or 16x16x64 int8 products, or one 16x16x128
// E4M3 product.  Weights are the A operand and token rows the B operand, so a lane ends up
// with four consecutive output columns of one token row.
#include "common.h"
#include "grouped.h"
#include "kernels.h"

namespace rmoe {

template <int Q>
using acc_t = typename AccOf<Q>::type;

// Token rows per tile of the streaming kernel, waves per workgroup.
constexpr int kStreamRows = 64, kStreamWaves = 4;

template <int Q, bool SITU, int WR>
__global__ __launch_bounds__(kStreamWaves * 64) void grouped_stream_kernel(GroupedArgs a) {
  extern __shared__ int32_t s_tile[];                  // [E + 1] first tile of each expert
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int g = lane >> 4, l16 = lane & 15;
  scan_tiles<kStreamRows, kStreamWaves>(a, s_tile);
  constexpr int kCols = kStreamWaves * WR * 16 / (SITU ? 2 : 1);   // output columns per item
  const int nblk = (a.N + kCols - 1) / kCols;
  const int64_t total = static_cast<int64_t>(s_tile[a.E]) * nblk;
  const int KB = a.KB, nc = (KB + 127) / 128;
  for (int64_t item = blockIdx.x; item < total; item += gridDim.x) {
    const int tile = static_cast<int>(item / nblk), cb = static_cast<int>(item % nblk);
    const TileRows tr = find_tile<kStreamRows>(a, s_tile, tile);
    // weight row of group r, MFMA row l16 (SiTU: even groups gate rows, odd groups the up
    // rows of the same columns); columns past N read the last row and are not stored
    const int c0 = cb * kCols + wave * (kCols / kStreamWaves);
    const uint8_t* wp[WR];
#pragma unroll
    for (int r = 0; r < WR; ++r) {
      const int n = min(c0 + 16 * (SITU ? r >> 1 : r) + l16, a.N - 1);
      const int64_t row = static_cast<int64_t>(tr.expert) * a.Nw + n + (SITU && (r & 1) ? a.N : 0);
      wp[r] = a.w + row * KB + 16 * g;
    }
    auto body = [&](auto mt_c) {
      constexpr int MT = decltype(mt_c)::value;
      const uint8_t* xp[MT];
      int64_t src[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        src[m] = 16 * m + l16 < tr.nrows ? source_row(a, tr.row0 + 16 * m + l16) : -1;
        xp[m] = a.x + src[m] * KB + 16 * g;
      }
      acc_t<Q> acc[WR][MT];
#pragma unroll
      for (int r = 0; r < WR; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[r][m] = acc_t<Q>{0, 0, 0, 0};
      for (int c = 0; c < nc; ++c) {
        u32x4 wv[WR][2], xv[MT][2];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const int off = 128 * c + 64 * f;
          const bool in = off + 16 * g < KB;
#pragma unroll
          for (int r = 0; r < WR; ++r) {
            wv[r][f] = u32x4{0, 0, 0, 0};
            if (in) wv[r][f] = *reinterpret_cast<const u32x4*>(wp[r] + off);
          }
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            xv[m][f] = u32x4{0, 0, 0, 0};
            if (in && src[m] >= 0) xv[m][f] = *reinterpret_cast<const u32x4*>(xp[m] + off);
          }
        }
#pragma unroll
        for (int r = 0; r < WR; ++r)
#pragma unroll
          for (int m = 0; m < MT; ++m)
            acc[r][m] = mma_chunk<Q>(wv[r][0], wv[r][1], xv[m][0], xv[m][1], acc[r][m]);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (16 * m + l16 >= tr.nrows) continue;
        uint16_t* orow = a.out + static_cast<int64_t>(tr.row0 + 16 * m + l16) * a.N;
        const float xs = Q == 0 || src[m] < 0 ? 1.0f : a.x_scale[src[m]];
#pragma unroll
        for (int r = 0; r < WR; r += SITU ? 2 : 1) {
          const int n0 = c0 + 16 * (SITU ? r >> 1 : r) + 4 * g;
          store4<Q, SITU>(a, tr.expert, n0, acc[r][m], acc[SITU ? r + 1 : r][m], xs, orow);
        }
      }
    };
    switch ((tr.nrows + 15) / 16) {
      case 1: body(IntC<1>{}); break;
      case 2: body(IntC<2>{}); break;
      case 3: body(IntC<3>{}); break;
      default: body(IntC<4>{}); break;
    }
  }
}

template <int Q, bool SITU>
static hipError_t launch_q(const GroupedArgs& a, hipStream_t stream) {
  constexpr int WR = 2;
  constexpr int kCols = kStreamWaves * WR * 16 / (SITU ? 2 : 1);
  const int64_t tiles = max_grouped_tiles(a.R, a.E, kStreamRows);
  const int64_t items = tiles * ((a.N + kCols - 1) / kCols);
  const int64_t slots = static_cast<int64_t>(a.cus) * 4;
  const unsigned grid = static_cast<unsigned>(items < slots ? items : slots);
  grouped_stream_kernel<Q, SITU, WR><<<dim3(grid), dim3(kStreamWaves * 64),
                                       (static_cast<size_t>(a.E) + 1) * 4, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_grouped(const GroupedArgs& a, hipStream_t stream) {
  switch (a.quant) {
    case 0: return a.situ ? launch_q<0, true>(a, stream) : launch_q<0, false>(a, stream);
    case 1: return a.situ ? launch_q<1, true>(a, stream) : launch_q<1, false>(a, stream);
    default: return a.situ ? launch_q<3, true>(a, stream) : launch_q<3, false>(a, stream);
  }
}

}  // namespace rmoe
