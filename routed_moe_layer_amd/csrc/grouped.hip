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
#pragma unroll
  for (int i = 0; i < PPT; ++i) {
    const int row = (tid + kMidThreads * i) / kPieces;
    // rows that are not there read the first of the tile; the epilogue leaves them out
    const int64_t src = source_row(a, tr.row0 + (row < tr.nrows ? row : 0));
    xp[i] = a.x + (src < 0 ? 0 : src) * KB + (tid % kPieces) * 16;
  }
  u32x4 xr[PPT], wv[kDepth][WR][2];
  auto load_x = [&](int s) {
    const int off = s * (CPS * 128);
#pragma unroll
    for (int i = 0; i < PPT; ++i) {
      xr[i] = u32x4{0, 0, 0, 0};
      if (off + (tid % kPieces) * 16 < KB)
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
  constexpr int C = SITU ? WR / 2 : WR;
  Epilogue<Q, SITU, C, MT> out(a);
  out.begin(tr.expert, [&](int c) { return c0 + 16 * c + 4 * g; },
            [&](int m) { return 16 * m + l16 < tr.nrows ? tr.row0 + 16 * m + l16 : -1; });
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if (out.row[m] < 0) continue;
#pragma unroll
    for (int c = 0; c < C; ++c)
      out.store(c, m, out.columns(c, m, acc[SITU ? 2 * c : c][m], acc[SITU ? 2 * c + 1 : c][m]));
  }
}

template <int Q, bool SITU>
__global__ __launch_bounds__(kMidThreads, 2) void grouped_mid_kernel(GroupedArgs a) {
  extern __shared__ int32_t s_tile[];
  __shared__ alignas(16) uint8_t stage[2 * kMidStageBytes];
  scan_experts<kMidWaves>(a, s_tile, [](int n) { return (n + kMidRows - 1) / kMidRows; });
  constexpr int kCols = kMidWaves * kMidWR * 16 / (SITU ? 2 : 1);
  const int nblk = (a.N + kCols - 1) / kCols;
  ItemWalk walk(a, s_tile, nblk);
  TileRows tr;
  int cb;
  while (walk.next<kMidRows>(&tr, &cb)) {
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

// ---------------------------------------------------------------------------------------
// Tiles of up to 256 rows for experts with many rows.  A workgroup of eight wavefronts
// multiplies 256 token rows with 256 weight rows, 128 x 64 per wavefront; both operands go
// from memory straight into LDS, one chunk of 128 bytes of K ahead, and are read as MFMA
// fragments from there.
// ---------------------------------------------------------------------------------------
constexpr int kBigTile = 256, kBigWaves = 8, kBigThreads = kBigWaves * 64;
constexpr int kBigOperandBytes = kBigTile * 128;

// Sixteen zero bytes: what a lane loads in the place of rows and columns that are not there.
__device__ const u32x4 g_zero16 = {0u, 0u, 0u, 0u};

typedef const __attribute__((address_space(1))) void* global_ptr;
typedef __attribute__((address_space(3))) void* lds_ptr;

// The wave's 64 x 16 bytes from each lane's address into consecutive LDS bytes.
__device__ __forceinline__ void load_to_lds(const uint8_t* src, uint8_t* dst) {
  __builtin_amdgcn_global_load_lds((global_ptr)src, (lds_ptr)dst, 16, 0, 0);
}

template <int Q, bool SITU>
__global__ __launch_bounds__(kBigThreads, 2) void grouped_big_kernel(GroupedArgs a) {
  extern __shared__ int32_t s_tile[];                  // two prefix sums of E + 1
  __shared__ alignas(16) uint8_t s_w0[kBigOperandBytes], s_x0[kBigOperandBytes];
  __shared__ alignas(16) uint8_t s_w1[kBigOperandBytes], s_x1[kBigOperandBytes];
  scan_experts<kBigWaves>(a, s_tile, [](int n) { return n / kBigTile; });
  scan_experts<kBigWaves>(a, s_tile + a.E + 1, [](int n) { return n % kBigTile != 0 ? 1 : 0; });
  constexpr int kCols = kBigTile / (SITU ? 2 : 1);
  const int nblk = (a.N + kCols - 1) / kCols;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int g = lane >> 4, l16 = lane & 15;
  // the wave's weight quarter and token half (the two waves of a SIMD have different halves)
  const int wn = wave & 3, wm = wave >> 2;
  const int KB = a.KB, nc = (KB + 127) / 128;
  const uint8_t* zero = reinterpret_cast<const uint8_t*>(&g_zero16);
  FullFirstWalk<kBigTile> walk(a, s_tile, s_tile + a.E + 1, nblk);

  // Load side: load j of a wave fills rows 32 wave + 8 j + lane / 8 of both operands, slot
  // lane % 8 of a row holding piece (lane % 8) ^ (row % 8): the eight rows that a fragment
  // read touches together fall on different banks.
  const uint8_t *wp[4], *xp[4];
  const int piece = ((lane & 7) ^ (lane >> 3)) * 16;
  TileRows ld;
  int ld_cb = 0, ld_c = 0;
  auto begin_item = [&]() {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = 32 * wave + 8 * j + (lane >> 3);
      // Row 64 q + 16 r + m holds the weights of MFMA row m of group r of the waves with
      // wn = q.  The order is chosen for the lanes' accumulators, four rows m = 4 g .. 4 g + 3
      // of each group: groups 2 s and 2 s + 1 make eight consecutive columns 32 s + 8 g + ...,
      // with SiTU groups 0 and 2 (gate) and 1 and 3 (up) columns 8 g + ....
      const int q = row >> 6, r = (row >> 4) & 3, m = row & 15;
      int n, up = 0;
      if (SITU) {
        n = ld_cb * kCols + 32 * q + 8 * (m >> 2) + 4 * (r >> 1) + (m & 3);
        up = r & 1;
      } else {
        n = ld_cb * kCols + 64 * q + 32 * (r >> 1) + 8 * (m >> 2) + 4 * (r & 1) + (m & 3);
      }
      n = min(n, a.N - 1) + (up ? a.N : 0);
      wp[j] = a.w + (static_cast<int64_t>(ld.expert) * a.Nw + n) * KB + piece;
      // rows that are not there read the first of the tile; the epilogue leaves them out
      const int64_t src = source_row(a, ld.row0 + (row < ld.nrows ? row : 0));
      xp[j] = a.x + (src < 0 ? 0 : src) * KB + piece;
    }
  };
  auto load = [&](uint8_t* sw, uint8_t* sx) {
    const int off = 128 * ld_c;
    const bool in = off + piece < KB;
#pragma unroll
    for (int j = 0; j < 4; ++j) load_to_lds(in ? wp[j] + off : zero, sw + (32 * wave + 8 * j) * 128);
    if (32 * wave < ld.nrows) {
#pragma unroll
      for (int j = 0; j < 4; ++j) load_to_lds(in ? xp[j] + off : zero, sx + (32 * wave + 8 * j) * 128);
    }
  };
  // The loads of the chunk after the one that was loaded last: the item's next, or the first
  // of the next item.  (An item has an even number of chunks, a last one of zeros where K has
  // an odd one, so that items start with the first buffers.)
  const int even = nc + (nc & 1);
  bool more = walk.next(&ld, &ld_cb);
  if (!more) return;
  auto load_next = [&](uint8_t* sw, uint8_t* sx) {
    if (++ld_c == even) {
      ld_c = 0;
      more = walk.next(&ld, &ld_cb);
      if (more) begin_item();
    }
    if (more) load(sw, sx);
  };

  // One item whose rows fit 32 MG tokens; a wave has 16 MG of them.
  auto item = [&](auto mg_c) {
    constexpr int MG = decltype(mg_c)::value;
    const int t0 = 16 * MG * wm;
    acc_t<Q> acc[4][MG];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int m = 0; m < MG; ++m) acc[r][m] = acc_t<Q>{0, 0, 0, 0};
    auto compute = [&](const uint8_t* sw, const uint8_t* sx) {
      u32x4 wf[4][2], xf[2][2];
      auto read_x = [&](int m) {
#pragma unroll
        for (int f = 0; f < 2; ++f)
          xf[m & 1][f] = *reinterpret_cast<const u32x4*>(
              sx + (t0 + 16 * m + l16) * 128 + (((4 * f + g) ^ (l16 & 7)) << 4));
      };
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int f = 0; f < 2; ++f)
          wf[r][f] = *reinterpret_cast<const u32x4*>(
              sw + (64 * wn + 16 * r + l16) * 128 + (((4 * f + g) ^ (l16 & 7)) << 4));
      read_x(0);
#pragma unroll
      for (int m = 0; m < MG; ++m) {
        if (m < MG - 1) read_x(m + 1);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[r][m] = mma_chunk<Q>(wf[r][0], wf[r][1], xf[m & 1][0], xf[m & 1][1], acc[r][m]);
      }
      if constexpr (MG == 8) {
        // issue order: the first reads, then each token group's reads one group ahead
        constexpr int kMfma = Q == 3 ? 4 : 8;
        __builtin_amdgcn_sched_group_barrier(0x100, 12, 0);
#pragma unroll
        for (int m = 0; m < 6; ++m) {
          __builtin_amdgcn_sched_group_barrier(0x008, kMfma, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, 2 * kMfma, 0);
      }
    };
    const TileRows tr = ld;
    const int cb = ld_cb;
    for (int c = 0; c < even; c += 2) {
      load_next(s_w1, s_x1);
      compute(s_w0, s_x0);
      __builtin_amdgcn_s_waitcnt(0);                   // this wave's loads are in LDS
      __syncthreads();
      load_next(s_w0, s_x0);
      compute(s_w1, s_x1);
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
    }
    constexpr int C = SITU ? 2 : 4;
    Epilogue<Q, SITU, C, MG> out(a);
    out.begin(
        tr.expert,
        [&](int n) {
          return cb * kCols + 8 * g + (SITU ? 32 * wn + 4 * n : 64 * wn + 32 * (n >> 1) + 4 * (n & 1));
        },
        [&](int m) {
          const int t = t0 + 16 * m + l16;
          return t < tr.nrows ? tr.row0 + t : -1;
        });
#pragma unroll
    for (int m = 0; m < MG; ++m) {
      if (out.row[m] < 0) continue;
#pragma unroll
      for (int n = 0; n < C; n += 2)
        out.store(n, m,
                  out.columns(n, m, acc[SITU ? 2 * n : n][m], acc[SITU ? 2 * n + 1 : n][m]),
                  out.columns(n + 1, m, acc[SITU ? 2 * n + 2 : n + 1][m],
                              acc[SITU ? 2 * n + 3 : n + 1][m]));
    }
  };

  begin_item();
  load(s_w0, s_x0);
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  while (more) {
    if (ld.nrows > 128) item(IntC<8>{});
    else if (ld.nrows > 64) item(IntC<4>{});
    else if (ld.nrows > 32) item(IntC<2>{});
    else item(IntC<1>{});
  }
}

template <int Q, bool SITU>
static hipError_t launch_big(const GroupedArgs& a, hipStream_t stream) {
  const unsigned grid = static_cast<unsigned>(a.cus / a.xcds * a.xcds);
  grouped_big_kernel<Q, SITU><<<dim3(grid), dim3(kBigThreads),
                                (static_cast<size_t>(a.E) + 1) * 8, stream>>>(a);
  return hipGetLastError();
}

template <int Q, bool SITU>
static hipError_t launch_one(const GroupedArgs& a, hipStream_t stream) {
  if (a.E <= 1024 && a.R >= a.E * 256) return launch_big<Q, SITU>(a, stream);
  return launch_mid<Q, SITU>(a, stream);
}

hipError_t launch_grouped(const GroupedArgs& a, hipStream_t stream) {
  switch (a.quant) {
    case 0: return a.situ ? launch_one<0, true>(a, stream) : launch_one<0, false>(a, stream);
    case 1: return a.situ ? launch_one<1, true>(a, stream) : launch_one<1, false>(a, stream);
    default: return a.situ ? launch_one<3, true>(a, stream) : launch_one<3, false>(a, stream);
  }
}

}  // namespace rmoe
