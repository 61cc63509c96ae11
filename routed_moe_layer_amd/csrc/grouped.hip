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

// ---------------------------------------------------------------------------------------
// Tiles of up to 128 rows.  A workgroup of four wavefronts multiplies one tile of an expert's
// rows with 128 weight rows, 32 per wavefront.  Each weight is used by one wavefront only, so
// weights go from memory to registers, kDepth chunks of 128 bytes ahead; the token rows are
// shared, so they pass through LDS in double-buffered stages of CPS chunks.
// ---------------------------------------------------------------------------------------
constexpr int kMidRows = 128, kMidWaves = 4, kMidThreads = kMidWaves * 64, kMidWR = 2;
constexpr int kMidStageBytes = 16384;
constexpr int kTileRun = 4;              // consecutive tiles kept on one XCD

template <int Q, bool SITU, int MT>
__device__ __forceinline__ void mid_tile(const GroupedArgs& a, const TileRows& tr, int cb,
                                         uint8_t* stage) {
  constexpr int WR = kMidWR, kDepth = 4;
  constexpr int CPS = MT <= 2 ? 4 : MT <= 4 ? 2 : 1;         // chunks per stage
  constexpr int kPieces = CPS * 8;                           // 16-byte pieces of a row per stage
  constexpr int PPT = MT * 16 * kPieces / kMidThreads;       // pieces per thread
  static_assert(MT * 16 * CPS * 128 <= kMidStageBytes && PPT * kMidThreads == MT * 16 * kPieces, "");
  constexpr int kCols = kMidWaves * WR * 16 / (SITU ? 2 : 1);
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int g = lane >> 4, l16 = lane & 15;
  const int KB = a.KB, nc = (KB + 127) / 128;
  const int c0 = cb * kCols + wave * (kCols / kMidWaves);
  const uint8_t* wp[WR];
#pragma unroll
  for (int r = 0; r < WR; ++r) {
    const int n = min(c0 + 16 * (SITU ? r >> 1 : r) + l16, a.N - 1);
    const int64_t row = static_cast<int64_t>(tr.expert) * a.Nw + n + (SITU && (r & 1) ? a.N : 0);
    wp[r] = a.w + row * KB + 16 * g;
  }
  // this thread's pieces of a stage: row q / kPieces, piece q % kPieces, q = tid + 256 i
  const uint8_t* xp[PPT];
  bool xok[PPT];
#pragma unroll
  for (int i = 0; i < PPT; ++i) {
    const int row = (tid + kMidThreads * i) / kPieces;
    const int64_t src = row < tr.nrows ? source_row(a, tr.row0 + row) : -1;
    xok[i] = src >= 0;
    xp[i] = a.x + (src < 0 ? 0 : src) * KB + (tid % kPieces) * 16;
  }
  u32x4 xr[PPT], wv[kDepth][WR][2];
  auto load_x = [&](int s) {
    const int off = s * (CPS * 128);
#pragma unroll
    for (int i = 0; i < PPT; ++i) {
      xr[i] = u32x4{0, 0, 0, 0};
      if (xok[i] && off + (tid % kPieces) * 16 < KB)
        xr[i] = *reinterpret_cast<const u32x4*>(xp[i] + off);
    }
  };
  // LDS stage: [chunk][row][8 pieces], a row's pieces permuted by its low three bits, so that
  // eight rows' reads of one piece fall on different banks
  auto store_x = [&](int s) {
    uint8_t* buf = stage + (s & 1) * kMidStageBytes;
#pragma unroll
    for (int i = 0; i < PPT; ++i) {
      const int q = tid + kMidThreads * i, row = q / kPieces, pc = q % kPieces;
      *reinterpret_cast<u32x4*>(buf + (pc >> 3) * (MT * 16 * 128) + row * 128 +
                                (((pc & 7) ^ (row & 7)) << 4)) = xr[i];
    }
  };
  auto load_w = [&](int u, int c) {
    const int off = 128 * c;
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int r = 0; r < WR; ++r) {
        if (off + 128 <= KB) {
          wv[u][r][f] = *reinterpret_cast<const u32x4*>(wp[r] + off + 64 * f);
        } else {
          wv[u][r][f] = u32x4{0, 0, 0, 0};
          if (off + 64 * f + 16 * g < KB)
            wv[u][r][f] = *reinterpret_cast<const u32x4*>(wp[r] + off + 64 * f);
        }
      }
  };
  acc_t<Q> acc[WR][MT];
#pragma unroll
  for (int r = 0; r < WR; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[r][m] = acc_t<Q>{0, 0, 0, 0};
  load_x(0);
#pragma unroll
  for (int u = 0; u < kDepth - 1; ++u)
    if (u < nc) load_w(u, u);
  store_x(0);
  __syncthreads();
  for (int cg = 0; cg < nc; cg += kDepth) {
#pragma unroll
    for (int u = 0; u < kDepth; ++u) {
      const int c = cg + u;
      if (c < nc) {
        const int s = c / CPS;
        if (u % CPS == 0) load_x(s + 1);
        if (c + kDepth - 1 < nc) load_w((u + kDepth - 1) % kDepth, c + kDepth - 1);
        const uint8_t* buf = stage + (s & 1) * kMidStageBytes + (u % CPS) * (MT * 16 * 128) + l16 * 128;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          u32x4 xv[2];
#pragma unroll
          for (int f = 0; f < 2; ++f)
            xv[f] = *reinterpret_cast<const u32x4*>(buf + m * 2048 + (((4 * f + g) ^ (l16 & 7)) << 4));
#pragma unroll
          for (int r = 0; r < WR; ++r)
            acc[r][m] = mma_chunk<Q>(wv[u][r][0], wv[u][r][1], xv[0], xv[1], acc[r][m]);
        }
        if (u % CPS == CPS - 1 || c == nc - 1) {
          store_x(s + 1);
          __syncthreads();
        }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if (16 * m + l16 >= tr.nrows) continue;
    const int i = tr.row0 + 16 * m + l16;
    uint16_t* orow = a.out + static_cast<int64_t>(i) * a.N;
    float xs = 1.0f;
    if constexpr (Q != 0) {
      const int64_t src = source_row(a, i);
      if (src >= 0) xs = a.x_scale[src];
    }
#pragma unroll
    for (int r = 0; r < WR; r += SITU ? 2 : 1) {
      const int n0 = c0 + 16 * (SITU ? r >> 1 : r) + 4 * g;
      store4<Q, SITU>(a, tr.expert, n0, acc[r][m], acc[SITU ? r + 1 : r][m], xs, orow);
    }
  }
}

template <int Q, bool SITU>
__global__ __launch_bounds__(kMidThreads, 2) void grouped_mid_kernel(GroupedArgs a) {
  extern __shared__ int32_t s_tile[];
  __shared__ alignas(16) uint8_t stage[2 * kMidStageBytes];
  scan_tiles<kMidRows, kMidWaves>(a, s_tile);
  constexpr int kCols = kMidWaves * kMidWR * 16 / (SITU ? 2 : 1);
  const int nblk = (a.N + kCols - 1) / kCols;
  const int tiles = s_tile[a.E];
  // XCD x takes runs of kTileRun consecutive tiles (tiles of one expert read the same
  // weights) and all their weight blocks (which read the same rows)
  const int xcd = static_cast<int>(blockIdx.x) % a.xcds, slot = static_cast<int>(blockIdx.x) / a.xcds;
  const int slots = static_cast<int>(gridDim.x) / a.xcds;
  const int64_t per_run = static_cast<int64_t>(kTileRun) * nblk;
  for (int64_t l = slot;; l += slots) {
    const int64_t run = l / per_run * a.xcds + xcd;
    if (run * kTileRun >= tiles) break;
    const int rem = static_cast<int>(l % per_run);
    const int tile = static_cast<int>(run * kTileRun) + rem % kTileRun;
    if (tile >= tiles) continue;
    const TileRows tr = find_tile_even<kMidRows>(a, s_tile, tile);
    const int cb = rem / kTileRun;
    if (tr.nrows <= 0) continue;
    const int mt = (tr.nrows + 15) / 16;
    if (mt <= 1) mid_tile<Q, SITU, 1>(a, tr, cb, stage);
    else if (mt <= 2) mid_tile<Q, SITU, 2>(a, tr, cb, stage);
    else if (mt <= 4) mid_tile<Q, SITU, 4>(a, tr, cb, stage);
    else if (mt <= 6) mid_tile<Q, SITU, 6>(a, tr, cb, stage);
    else mid_tile<Q, SITU, 8>(a, tr, cb, stage);
  }
}

template <int Q, bool SITU>
static hipError_t launch_mid(const GroupedArgs& a, hipStream_t stream) {
  const unsigned grid = static_cast<unsigned>(a.cus / a.xcds * a.xcds * 2);
  grouped_mid_kernel<Q, SITU><<<dim3(grid), dim3(kMidThreads), (static_cast<size_t>(a.E) + 1) * 4,
                                stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_grouped(const GroupedArgs& a, hipStream_t stream) {
  switch (a.quant) {
    case 0: return a.situ ? launch_mid<0, true>(a, stream) : launch_mid<0, false>(a, stream);
    case 1: return a.situ ? launch_mid<1, true>(a, stream) : launch_mid<1, false>(a, stream);
    default: return a.situ ? launch_mid<3, true>(a, stream) : launch_mid<3, false>(a, stream);
  }
}

}  // namespace rmoe
