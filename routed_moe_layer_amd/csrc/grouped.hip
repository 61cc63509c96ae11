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
#include <algorithm>

#include "common.h"
#include "grouped.h"
#include "kernels.h"

namespace rmoe {

template <int Q>
using acc_t = typename AccOf<Q>::type;

// ---------------------------------------------------------------------------------------
// Tiles of up to BM rows (32, 64 or 128).  A workgroup of NW wavefronts multiplies one tile of
// an expert's rows with 32 NW weight rows, 32 per wavefront.  Both operands go from memory
// straight into LDS in chunks of 128 bytes of K, in a ring of S chunks that runs on over the
// border between two items.  Every wavefront issues the same number of loads per chunk, so
// one counted wait per chunk is enough: a chunk is there when no more loads are under way than
// were issued after it.
//
// Bound by the bytes of the weights: FC1 of 16 tokens over 896 experts (BF16, N = 384 with
// SiTU, K = 3584, 1.24 GB) 214 us, 5.8 TB/s; FC2 of 1024 Zipf tokens (N = 3584, K = 384, 2.55
// GB) 481 us, 5.3 TB/s; FC1 of 4096 tokens in int8 (2.53 GB) 507 us, 5.0 TB/s; a large read on
// the same card 5.99 TB/s.  Weights in registers instead of LDS (each is used by one wavefront)
// and token rows through registers took 238, 602 and 638 us: loads complete in order, so the
// wait for a chunk's token rows was one for the weights loaded ahead of them too.
// ---------------------------------------------------------------------------------------
template <int Q, bool SITU, int BM, int NW, int PER_CU, int S>
__global__ __launch_bounds__(NW * 64, NW * PER_CU / 4) void grouped_mid_kernel(GroupedArgs a) {
  constexpr int kRows = 32 * NW, kCols = kRows / (SITU ? 2 : 1);
  constexpr int kXLoads = BM / (8 * NW), kLoads = 4 + kXLoads;       // per wavefront and chunk
  static_assert(kXLoads * 8 * NW == BM, "");
  extern __shared__ int32_t s_tile[];
  // the ring's buffers: arrays of their own, so that the compiler sees which loads into LDS a
  // read has to wait for (none, after the counted wait); weights, then token rows
  __shared__ alignas(16) uint8_t s_0[(kRows + BM) * 128], s_1[(kRows + BM) * 128],
      s_2[(kRows + BM) * 128];
  auto ring = [&](auto u) {
    constexpr int U = decltype(u)::value % S;
    if constexpr (U == 0) return &s_0[0];
    else if constexpr (U == 1) return &s_1[0];
    else if constexpr (U == 2) return &s_2[0];
    else return more_ring<U, (kRows + BM) * 128>();
  };
  scan_experts<NW>(a, s_tile, a.R / BM + min(a.R, a.E), [](int n) { return (n + BM - 1) / BM; });
  const int nblk = (a.N + kCols - 1) / kCols;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int g = lane >> 4, l16 = lane & 15;
  const int KB = a.KB;
  // an item takes whole rounds of the ring (chunks past the end of K are zeros), so that every
  // item starts with the first buffers
  const int nc = (KB + 128 * S - 1) / (128 * S) * S;
  const uint8_t* zero = reinterpret_cast<const uint8_t*>(&g_zero16);
  ItemWalk walk(a, s_tile, nblk);
  TileRows ld;
  int ld_cb = 0;
  bool more = walk.next<BM>(&ld, &ld_cb);
  if (!more) return;                                   // the whole workgroup

  // Load j of a wavefront fills rows 8 j + lane / 8 of its 32 weight rows, or of its token
  // rows; slot lane % 8 of a row holds piece (lane % 8) ^ (row % 8), so that eight rows' reads
  // of one piece fall on different banks.
  const uint8_t *wp[4], *xp[kXLoads];
  const int piece = ((lane & 7) ^ (lane >> 3)) * 16;
  auto begin_item = [&]() {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // LDS row 16 r + m holds MFMA row m of group r: columns 8 (m / 4) + 4 r + m % 4 of the
      // wavefront's 32, so that a lane's two groups make eight consecutive columns; with SiTU
      // column m, the gate row in group 0 and the up row in group 1
      const int l8 = lane >> 3, r = j >> 1, m = 8 * (j & 1) + l8;
      const int n = ld_cb * kCols + wave * (kCols / NW) +
                    (SITU ? m : 8 * (m >> 2) + 4 * r + (m & 3));
      const int64_t row = static_cast<int64_t>(ld.expert) * a.Nw + min(n, a.N - 1);
      wp[j] = a.w + (row + (SITU && r ? a.N : 0)) * KB + piece;
    }
#pragma unroll
    for (int j = 0; j < kXLoads; ++j) {
      const int row = 8 * (NW * j + wave) + (lane >> 3);
      // rows that are not there read the first of the tile; the epilogue leaves them out
      const int64_t src = source_row(a, ld.row0 + (row < ld.nrows ? row : 0));
      xp[j] = a.x + (src < 0 ? 0 : src) * KB + piece;
    }
  };
  auto load = [&](uint8_t* buf, int c) {
    uint8_t* sx = buf + kRows * 128;
    const int off = 128 * c;
    const bool in = off + piece < KB;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      load_to_lds(in ? wp[j] + off : zero, buf + (32 * wave + 8 * j) * 128);
#pragma unroll
    for (int j = 0; j < kXLoads; ++j)
      load_to_lds(in ? xp[j] + off : zero, sx + 8 * (NW * j + wave) * 128);
  };

  auto item = [&](auto mt_c, const TileRows tr, const int cb) {
    constexpr int MT = decltype(mt_c)::value;
    acc_t<Q> acc[2][MT];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[r][m] = acc_t<Q>{0, 0, 0, 0};
    // this wavefront's loads of the chunk are in LDS, and it is done reading the buffers that
    // the next loads write; after the barrier that holds for the workgroup
    auto arrive = [&]() {
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(wait_vm_lds((S - 2) * kLoads));
      asm volatile("s_barrier" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    };
    auto compute = [&](const uint8_t* sw) {
      const uint8_t* sx = sw + kRows * 128;
      u32x4 wf[2][2];
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int f = 0; f < 2; ++f)
          wf[r][f] = *reinterpret_cast<const u32x4*>(sw + (32 * wave + 16 * r + l16) * 128 +
                                                     (((4 * f + g) ^ (l16 & 7)) << 4));
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        u32x4 xf[2];
#pragma unroll
        for (int f = 0; f < 2; ++f)
          xf[f] = *reinterpret_cast<const u32x4*>(sx + (16 * m + l16) * 128 +
                                                  (((4 * f + g) ^ (l16 & 7)) << 4));
#pragma unroll
        for (int r = 0; r < 2; ++r)
          acc[r][m] = mma_chunk<Q>(wf[r][0], wf[r][1], xf[0], xf[1], acc[r][m]);
      }
    };
    for (int c = 0; c < nc; c += S) {
      const bool last = c + S == nc;
      for_ring<S>([&](auto u) {
        constexpr int U = decltype(u)::value;
        arrive();
        // after an item's last chunk the first of the next item, or of this one again behind
        // the last item, so that the number of loads under way stays the same
        if constexpr (U == 1) {
          if (last) {
            more = walk.next<BM>(&ld, &ld_cb);
            if (more) begin_item();
          }
        }
        load(ring(IntC<U + S - 1>{}), U > 0 && last ? U - 1 : c + U + S - 1);
        compute(ring(u));
      });
    }
    constexpr int C = SITU ? 1 : 2;
    Epilogue<Q, SITU, C, MT> out(a);
    const int n0 = cb * kCols + wave * (kCols / NW);
    out.begin(tr.expert, [&](int n) { return n0 + (SITU ? 4 * g : 8 * g + 4 * n); },
              [&](int m) { return 16 * m + l16 < tr.nrows ? tr.row0 + 16 * m + l16 : -1; });
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (out.row[m] < 0) continue;
      if constexpr (SITU)
        out.store(0, m, out.columns(0, m, acc[0][m], acc[1][m]));
      else
        out.store(0, m, out.columns(0, m, acc[0][m], acc[0][m]),
                  out.columns(1, m, acc[1][m], acc[1][m]));
    }
  };

  begin_item();
  TileRows tr = ld;
  int cb = ld_cb;
  // The load side is S - 1 chunks ahead: it is in the item that the other side begins.
  for_ring<S - 1>([&](auto u) { load(ring(u), decltype(u)::value); });
  for (;;) {
    const int mt = (tr.nrows + 15) / 16;
    if (mt <= 1) item(IntC<1>{}, tr, cb);
    else if (mt <= 2) item(IntC<2>{}, tr, cb);
    else if (BM == 64 || mt <= 4) item(IntC<BM >= 64 ? 4 : 2>{}, tr, cb);
    else if (mt <= 6) item(IntC<BM >= 128 ? 6 : 2>{}, tr, cb);
    else item(IntC<BM >= 128 ? 8 : 2>{}, tr, cb);
    if (!more) break;
    tr = ld;
    cb = ld_cb;
  }
  __builtin_amdgcn_s_waitcnt(0);                       // no load into LDS outlives the workgroup
}

template <int Q, bool SITU, int BM, int NW, int PER_CU, int S>
static hipError_t launch_mid(const GroupedArgs& a, hipStream_t stream) {
  const unsigned grid = static_cast<unsigned>(a.cus / a.xcds * a.xcds * PER_CU);
  grouped_mid_kernel<Q, SITU, BM, NW, PER_CU, S>
      <<<dim3(grid), dim3(NW * 64), (static_cast<size_t>(a.E) + 1) * 4, stream>>>(a);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------------------
// Tiles of up to 256 rows for experts with many rows.  A workgroup of eight wavefronts
// multiplies 256 token rows with 256 weight rows, 128 x 64 per wavefront; both operands go
// from memory straight into LDS, one chunk of 128 bytes of K ahead (the two buffers of 64 KB
// fill the LDS), and are read as MFMA fragments from there.
//
// Bound by the matrix units and what surrounds them: 8 experts x 4096 rows in E4M3 (N = 3584,
// K = 4096) take 455 us, 2.1 PFLOP/s; their products alone, seven to eight rounds of items,
// 250 us at the clock the card holds; the same kernel without its stores 391 us.  One expert,
// 8192^3: E4M3 2.7, int8 2.1, BF16 1.3 PFLOP/s (large library products 2.5, 2.1 and 1.4).
// With the item loop and the K loop in one (an epilogue inside) the accumulators spilled.
// ---------------------------------------------------------------------------------------
constexpr int kBigTile = 256, kBigWaves = 8, kBigThreads = kBigWaves * 64;
constexpr int kBigOperandBytes = kBigTile * 128;

template <int Q, bool SITU>
__global__ __launch_bounds__(kBigThreads, 2) void grouped_big_kernel(GroupedArgs a) {
  extern __shared__ int32_t s_tile[];                  // two prefix sums of E + 1
  __shared__ alignas(16) uint8_t s_w0[kBigOperandBytes], s_x0[kBigOperandBytes];
  __shared__ alignas(16) uint8_t s_w1[kBigOperandBytes], s_x1[kBigOperandBytes];
  scan_experts<kBigWaves>(a, s_tile, a.R / kBigTile, [](int n) { return n / kBigTile; });
  scan_experts<kBigWaves>(a, s_tile + a.E + 1, 2 * min(a.R, a.E), [](int n) {
    return (n % kBigTile + kBigTile / 2 - 1) / (kBigTile / 2);
  });
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

// Which kernel.  Larger tiles read the weights for more rows at once; smaller ones and smaller
// blocks of weight rows make more work items.  items() is an upper bound of the items of a
// kernel (the host does not know the rows of each expert), `few` three quarters of the CUs.
// Measured on one MI355X, BF16 unless said otherwise, us with tiles of 256 / 128 / 64 / 32 rows:
//   many rows per expert: 64 experts x 512 rows, N = 768, K = 3584  238 / 242 / 299 / -, but
//     x 256 rows (half of the experts above one tile) 208 / 130 / 174 / -;
//   the same with too few items: one expert, 512 rows, N = K = 7168  151 / 89 / 69 / 112;
//   few rows, many items: FC2 of 1024 Zipf tokens over 896 experts, N = 3584, K = 384
//     - / 482 / 505 / 602;
//   few rows, few items: 8 experts x 32 rows, N = K = 4096  - / 54 / 46 / 60;
//     one expert, 64 rows, N = K = 7168  - / 59 / 41 / 26; one token's 16 experts, N = 384 with
//     SiTU, K = 3584  37 with blocks of 128 weight rows and 3 chunks, 22 with 64 and 6, whose
//     longer ring loses on short K (FC2 of 16 tokens over 896 experts, K = 384: 115 and 139).
template <int Q, bool SITU>
static hipError_t launch_one(const GroupedArgs& a, hipStream_t stream) {
  const int64_t R = a.R, E = a.E, few = a.cus * 3 / 4;
  auto items = [&](int tile, int block) {
    return (std::min(R, E) + R / tile) * ((a.Nw + block - 1) / block);
  };
  // (the LDS of the two largest tiles leaves room for so many experts' prefix sums)
  if (E <= 1024 && R >= 448 * E && items(256, 256) >= few) return launch_big<Q, SITU>(a, stream);
  const int64_t items128 = items(128, 256);
  if (E <= 2048 && (items128 >= 8 * a.cus || (R > 40 * E && items128 >= few)))
    return launch_mid<Q, SITU, 128, 8, 1, 3>(a, stream);
  if (R > 24 * E && items(64, 128) >= few) return launch_mid<Q, SITU, 64, 4, 2, 3>(a, stream);
  if (a.KB >= 2048) return launch_mid<Q, SITU, 32, 2, 2, 6>(a, stream);
  return launch_mid<Q, SITU, 32, 4, 2, 3>(a, stream);
}

hipError_t launch_grouped(const GroupedArgs& a, hipStream_t stream) {
  switch (a.quant) {
    case 0: return a.situ ? launch_one<0, true>(a, stream) : launch_one<0, false>(a, stream);
    case 1: return a.situ ? launch_one<1, true>(a, stream) : launch_one<1, false>(a, stream);
    default: return a.situ ? launch_one<3, true>(a, stream) : launch_one<3, false>(a, stream);
  }
}

}  // namespace rmoe
