// Matrix products grouped by expert with ragged sizes, both operands in microscaled FP4 (blocks
// of 32 along K with one E8M0 scale each):
//   h[i, n] = sum_b 2^(sx - 127) 2^(sw - 127) sum_{32} x * w,
//   out[i, n] = BF16(h[i, n])   or   BF16(SiTU(h[i, n], h[i, N + n]))  with Nw = 2N.
//
// The scaled matrix instruction does the whole of it: an operand fragment of 16x16x128 is 16
// bytes per lane (lane l: row l % 16, one block of 32), with the block's scale byte in a register
// of the lane.  It adds a block's products exactly and the blocks in fp32, applies the scales to
// the exponent (nothing underflows before fp32 does) and makes a NaN of a scale byte 255.
// Weights are the A operand and token rows the B operand, so a lane ends up with four consecutive
// output columns of one token row.
//
// A K chunk is 128 bytes of codes per row, eight blocks and two dwords of scales.  Its order in K
// is free as long as both operands agree: fragment f of lane group g takes block 2 g + f, so that
// a lane's two scale bytes lie next to each other and the instruction's byte selector is f.
#include <algorithm>

#include "common.h"
#include "grouped.h"
#include "kernels.h"

namespace rmoe {

// acc += A * B over one fragment each; F: which byte of the lanes' scales.
template <int F>
__device__ __forceinline__ f32x4 mx_mma(u32x4 a, u32x4 b, f32x4 acc, uint32_t sa, uint32_t sb) {
  i32x8 x = {0, 0, 0, 0, 0, 0, 0, 0}, y = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = static_cast<int>(a[i]);
    y[i] = static_cast<int>(b[i]);
  }
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc, 4, 4, F, static_cast<int>(sa),
                                                          F, static_cast<int>(sb));
}

// ---------------------------------------------------------------------------------------
// Tiles of up to BM rows (32, 64 or 128).  A workgroup of NW wavefronts multiplies one tile of
// an expert's rows with 32 NW weight rows, 32 per wavefront.  Codes and scales of both operands
// go from memory straight into LDS in chunks, in a ring of S chunks that runs on over the border
// between two items.  Every wavefront issues the same number of loads per chunk (the token rows'
// scales are loaded by several wavefronts alike), so one counted wait per chunk is enough: a
// chunk is there when no more loads are under way than were issued after it.
// ---------------------------------------------------------------------------------------
template <bool SITU, int BM, int NW, int PER_CU, int S>
__global__ __launch_bounds__(NW * 64, NW * PER_CU / 4) void grouped_mx_mid_kernel(MxGroupedArgs a) {
  constexpr int kRows = 32 * NW, kCols = kRows / (SITU ? 2 : 1);
  constexpr int kXLoads = BM / (8 * NW), kLoads = 6 + kXLoads;       // per wavefront and chunk
  static_assert(kXLoads * 8 * NW == BM && BM / 32 <= NW, "");
  // a buffer: weights, token rows, the weights' scales, the token rows' scales
  constexpr int kScales = (kRows + BM) * 128, kBytes = (kRows + BM) * 136;
  extern __shared__ int32_t s_tile[];
  __shared__ alignas(16) uint8_t s_0[kBytes], s_1[kBytes], s_2[kBytes];
  auto ring = [&](auto u) {
    constexpr int U = decltype(u)::value % S;
    if constexpr (U == 0) return &s_0[0];
    else if constexpr (U == 1) return &s_1[0];
    else if constexpr (U == 2) return &s_2[0];
    else return more_ring<U, kBytes>();
  };
  scan_experts<NW>(a, s_tile, a.R / BM + min(a.R, a.E), [](int n) { return (n + BM - 1) / BM; });
  const int nblk = (a.N + kCols - 1) / kCols;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int g = lane >> 4, l16 = lane & 15;
  const int KB = a.KB, SB = a.SB;
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
  // of one piece fall on different banks.  A load of scales takes 32 rows, two lanes each.
  const uint8_t *wp[4], *xp[kXLoads], *wsp, *xsp;
  const int piece = ((lane & 7) ^ (lane >> 3)) * 16, half = (lane & 1) * 4;
  const int xs_row = 32 * (wave % (BM / 32)) + (lane >> 1);
  // LDS row 16 r + m of a wavefront's weights holds MFMA row m of group r: columns 8 (m / 4) +
  // 4 r + m % 4 of its 32, so that a lane's two groups make eight consecutive columns; with SiTU
  // column m, the gate row in group 0 and the up row in group 1
  auto weight_row = [&](int i) {
    const int r = i >> 4, m = i & 15;
    const int n = ld_cb * kCols + wave * (kCols / NW) + (SITU ? m : 8 * (m >> 2) + 4 * r + (m & 3));
    return static_cast<int64_t>(ld.expert) * a.Nw + min(n, a.N - 1) + (SITU && r ? a.N : 0);
  };
  // rows that are not there read the first of the tile; the epilogue leaves them out
  auto token_row = [&](int i) {
    const int64_t src = source_row(a, ld.row0 + (i < ld.nrows ? i : 0));
    return src < 0 ? 0 : src;
  };
  auto begin_item = [&]() {
#pragma unroll
    for (int j = 0; j < 4; ++j) wp[j] = a.w + weight_row(8 * j + (lane >> 3)) * KB + piece;
    wsp = a.w_mx + weight_row(lane >> 1) * SB + half;
#pragma unroll
    for (int j = 0; j < kXLoads; ++j)
      xp[j] = a.x + token_row(8 * (NW * j + wave) + (lane >> 3)) * KB + piece;
    xsp = a.x_mx + token_row(xs_row) * SB + half;
  };
  auto load = [&](uint8_t* buf, int c) {
    const int off = 128 * c, soff = 8 * c;
    const bool in = off + piece < KB, s_in = soff + half < SB;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      load_to_lds(in ? wp[j] + off : zero, buf + (32 * wave + 8 * j) * 128);
#pragma unroll
    for (int j = 0; j < kXLoads; ++j)
      load_to_lds(in ? xp[j] + off : zero, buf + (kRows + 8 * (NW * j + wave)) * 128);
    load4_to_lds(s_in ? wsp + soff : zero, buf + kScales + 32 * wave * 8);
    load4_to_lds(s_in ? xsp + soff : zero, buf + kScales + (kRows + 32 * (wave % (BM / 32))) * 8);
  };

  auto item = [&](auto mt_c, const TileRows tr, const int cb) {
    constexpr int MT = decltype(mt_c)::value;
    f32x4 acc[2][MT];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[r][m] = f32x4{0, 0, 0, 0};
    // this wavefront's loads of the chunk are in LDS, and it is done reading the buffers that
    // the next loads write; after the barrier that holds for the workgroup
    auto arrive = [&]() {
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(wait_vm_lds((S - 2) * kLoads));
      asm volatile("s_barrier" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    };
    auto compute = [&](const uint8_t* buf) {
      auto fragment = [&](int row, int f) {
        return *reinterpret_cast<const u32x4*>(buf + row * 128 + (((2 * g + f) ^ (l16 & 7)) << 4));
      };
      auto scales = [&](int row) -> uint32_t {
        return *reinterpret_cast<const uint16_t*>(buf + kScales + row * 8 + 2 * g);
      };
      u32x4 wf[2][2];
      uint32_t ws[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        ws[r] = scales(32 * wave + 16 * r + l16);
#pragma unroll
        for (int f = 0; f < 2; ++f) wf[r][f] = fragment(32 * wave + 16 * r + l16, f);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int row = kRows + 16 * m + l16;
        const u32x4 x0 = fragment(row, 0), x1 = fragment(row, 1);
        const uint32_t xs = scales(row);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          acc[r][m] = mx_mma<0>(wf[r][0], x0, acc[r][m], ws[r], xs);
          acc[r][m] = mx_mma<1>(wf[r][1], x1, acc[r][m], ws[r], xs);
        }
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
    Epilogue<0, SITU, C, MT> out(a);
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

template <bool SITU, int BM, int NW, int PER_CU, int S>
static hipError_t launch_mx_mid(const MxGroupedArgs& a, hipStream_t stream) {
  const unsigned grid = static_cast<unsigned>(a.cus / a.xcds * a.xcds * PER_CU);
  grouped_mx_mid_kernel<SITU, BM, NW, PER_CU, S>
      <<<dim3(grid), dim3(NW * 64), (static_cast<size_t>(a.E) + 1) * 4, stream>>>(a);
  return hipGetLastError();
}

template <bool SITU>
static hipError_t launch_mx_one(const MxGroupedArgs& a, hipStream_t stream) {
  const int64_t R = a.R, E = a.E, few = a.cus * 3 / 4;
  auto items = [&](int tile, int block) {
    return (std::min(R, E) + R / tile) * ((a.Nw + block - 1) / block);
  };
  const int64_t items128 = items(128, 256);
  if (E <= 1536 && (items128 >= 8 * a.cus || (R > 40 * E && items128 >= few)))
    return launch_mx_mid<SITU, 128, 8, 1, 3>(a, stream);
  if (R > 24 * E && items(64, 128) >= few) return launch_mx_mid<SITU, 64, 4, 2, 3>(a, stream);
  if (a.KB >= 1024) return launch_mx_mid<SITU, 32, 2, 2, 6>(a, stream);
  return launch_mx_mid<SITU, 32, 4, 2, 3>(a, stream);
}

hipError_t launch_grouped_mxfp4(const MxGroupedArgs& a, hipStream_t stream) {
  return a.situ ? launch_mx_one<true>(a, stream) : launch_mx_one<false>(a, stream);
}

}  // namespace rmoe
