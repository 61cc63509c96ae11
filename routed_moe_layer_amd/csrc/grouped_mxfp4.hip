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

// A row's 16-byte pieces lie in the eight slots of its 128 bytes of LDS, piece p in slot
// p ^ mx_swizzle(row).  A fragment read takes pieces 2 g + f of sixteen rows; the LDS serves it in
// quarters of rows 0-3 and 12-15 of one lane group with rows 4-11 of the next (or the other way
// round), two rows side by side in its 64 banks.  With the row's bits 0 and 1 exchanged the
// sixteen lanes fall on different banks; with the row itself pieces 0 and 2 meet.
__device__ __forceinline__ int mx_swizzle(int row) {
  return (row & 4) | (row & 1) << 1 | (row >> 1 & 1);
}

// What a sorted row without a source reads: zeros for all of K, codes and scales.
__device__ const u32x4 g_zero_row[65536 / 2 / 16] = {};

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

// The same with the accumulator in place in AGPRs.  The builtin's result may go to other registers
// than its addend: with 256 of them in use that took 300 register moves per 256 products, and
// spills.  Written out, the instruction's waits are not the compiler's: an operand must not come
// from a vector instruction right before it (ready()), and a result must not be read by another
// kind of instruction before settle().
template <int F>
__device__ __forceinline__ void mx_mma_in_place(u32x4 a, u32x4 b, f32x4& acc, uint32_t sa, uint32_t sb) {
#define RMOE_MX_MMA(SEL)                                                                         \
  asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 " SEL        \
               " cbsz:4 blgp:4" : "+a"(acc) : "v"(a), "v"(b), "v"(sa), "v"(sb))
  if constexpr (F == 0) RMOE_MX_MMA("op_sel:[0,0,0] op_sel_hi:[0,0,0]");
  else if constexpr (F == 1) RMOE_MX_MMA("op_sel:[1,1,0] op_sel_hi:[0,0,0]");
  else if constexpr (F == 2) RMOE_MX_MMA("op_sel:[0,0,0] op_sel_hi:[1,1,0]");
  else RMOE_MX_MMA("op_sel:[1,1,0] op_sel_hi:[1,1,0]");
#undef RMOE_MX_MMA
}
// Eight consecutive columns n .. n + 7 of a row at o, those below N.  Where N is no multiple of 8 a
// row's columns are aligned to four or to one of them.
__device__ __forceinline__ void store_columns(uint16_t* o, u32x4 v, int N, int n) {
  if (N % 8 == 0 && n < N) {
    *reinterpret_cast<u32x4*>(o) = v;
  } else if (N % 4 == 0) {
    if (n < N) *reinterpret_cast<uint2*>(o) = make_uint2(v[0], v[1]);
    if (n + 4 < N) *reinterpret_cast<uint2*>(o + 4) = make_uint2(v[2], v[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (n + i < N) o[i] = static_cast<uint16_t>(v[i >> 1] >> (16 * (i & 1)));
  }
}

// Before a batch of them whose operands vector instructions may have written, two wait states.
// (Inside a batch only LDS reads write operands, which are waited for.  An s_nop in front of each
// instruction took 4% of 8192^3.)
__device__ __forceinline__ void ready() { asm volatile("s_nop 1" ::: "memory"); }
// Behind the last of them in a loop, before its branch: a 4-pass instruction's result is there
// after 7 wait states, and code behind the loop may read it at once.
__device__ __forceinline__ void settle() { asm volatile("s_nop 7" ::: "memory"); }

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

  // Load j of a wavefront fills rows 8 j + lane / 8 of its 32 weight rows, or of its token rows,
  // slot lane % 8 of a row with piece (lane % 8) ^ mx_swizzle(row).  A load of scales takes 32
  // rows, two lanes each.
  const uint8_t *wp[4], *xp[kXLoads], *wsp, *xsp;
  const int piece = ((lane & 7) ^ mx_swizzle(lane >> 3)) * 16, half = (lane & 1) * 4;
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
        return *reinterpret_cast<const u32x4*>(buf + row * 128 + (((2 * g + f) ^ mx_swizzle(l16)) << 4));
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

// ---------------------------------------------------------------------------------------
// Tiles of up to 256 rows for experts with many rows.  A workgroup of four wavefronts multiplies
// 256 token rows with 256 weight rows, 128 x 128 per wavefront.  Both operands go from memory
// straight into LDS in chunks of 128 bytes per row (whole cache lines: half of them per load made
// twice the requests and took a fifth more time), two buffers of 32 KB each.  A chunk is two
// steps of one fragment each.  The weights' fragments of a step are read into registers during
// the step before, so a chunk's weights leave their buffer after its first step and its token rows
// after the second: the weights of the chunk after the next are loaded in the second step, the
// next chunk's token rows in the first, and both have two steps' time.
//
// Scales come in rounds of two chunks, 16 bytes per row, through registers, where the pairs of
// bytes are transposed so that a lane reads one dword per row and round and a step is a byte
// selector of the instruction.
//
// Bound by the matrix units, the LDS and the caches together and by the power they draw: 8192^3
// takes 251 us, 4.4 PFLOP/s (the instruction alone on random codes 6.7, with the clock down to
// 1.6 GHz; the same kernel without its loads 4.6, without its LDS reads 4.7; the library's product
// 2.9).  8 experts x 4096 rows (N = 3584, K = 4096) take 276 us, 3.5 PFLOP/s, in seven to eight
// rounds of items.  Eight wavefronts of 128 x 64 products read 1.5 times as much from LDS.
// ---------------------------------------------------------------------------------------
constexpr int kWaitLds = 0xC07F;                       // s_waitcnt for LDS reads alone
constexpr int kMxTile = 256, kMxWaves = 4, kMxThreads = kMxWaves * 64;
constexpr int kMxBufBytes = kMxTile * 128, kMxBufLoads = kMxBufBytes / 1024 / kMxWaves;

template <bool SITU>
__global__ __launch_bounds__(kMxThreads, 1) void grouped_mx_big_kernel(MxGroupedArgs a) {
  extern __shared__ int32_t s_tile[];                  // two prefix sums of E + 1
  __shared__ alignas(16) uint8_t s_w0[kMxBufBytes], s_w1[kMxBufBytes], s_x0[kMxBufBytes],
      s_x1[kMxBufBytes];
  __shared__ alignas(16) u32x4 s_scale[2 * kMxTile];
  scan_experts<kMxWaves>(a, s_tile, a.R / kMxTile, [](int n) { return n / kMxTile; });
  scan_experts<kMxWaves>(a, s_tile + a.E + 1, 2 * min(a.R, a.E), [](int n) {
    return (n % kMxTile + kMxTile / 2 - 1) / (kMxTile / 2);
  });
  constexpr int kCols = kMxTile / (SITU ? 2 : 1);
  const int nblk = (a.N + kCols - 1) / kCols;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int g = lane >> 4, l16 = lane & 15;
  const int wn = wave & 1, wm = wave >> 1;             // the wave's weight half and token half
  const int KB = a.KB, SB = a.SB;
  const int nr = (KB + 255) / 256;                     // rounds of two chunks
  const uint8_t *zero = reinterpret_cast<const uint8_t*>(&g_zero16),
                *zeros = reinterpret_cast<const uint8_t*>(g_zero_row);
  FullFirstWalk<kMxTile> walk(a, s_tile, s_tile + a.E + 1, nblk);
  TileRows ld;
  int ld_cb = 0, ld_r = 0;
  bool more = walk.next(&ld, &ld_cb);
  if (!more) return;                                   // the whole workgroup

  // Weight row of LDS row i: row 128 q + 16 r + m holds the weights of MFMA row m of group r of
  // the waves with wn = q.  The order is chosen for the lanes' accumulators, four rows m = 4 g ..
  // 4 g + 3 of each group: groups 2 s and 2 s + 1 make eight consecutive columns 32 s + 8 g + ...,
  // with SiTU groups 4 s and 4 s + 2 (gate) and the ones behind them (up).
  auto weight_row = [&](int i) {
    const int q = i >> 7, r = (i >> 4) & 7, m = i & 15;
    int n;
    if (SITU) n = ld_cb * kCols + 64 * q + 32 * (r >> 2) + 8 * (m >> 2) + 4 * ((r >> 1) & 1) + (m & 3);
    else n = ld_cb * kCols + 128 * q + 32 * (r >> 1) + 8 * (m >> 2) + 4 * (r & 1) + (m & 3);
    return static_cast<int64_t>(ld.expert) * a.Nw + min(n, a.N - 1) + (SITU && (r & 1) ? a.N : 0);
  };
  // source row of token row i, -1 for zeros; rows that are not there read the first of the tile,
  // and the epilogue leaves them out
  auto token_row = [&](int i) { return source_row(a, ld.row0 + (i < ld.nrows ? i : 0)); };
  // Load j of a wave fills rows 64 wave + 8 j + lane / 8 of an operand, slot lane % 8 of a row
  // with piece (lane % 8) ^ mx_swizzle(row).  Thread t loads the scales of row t of both operands.
  const uint8_t *wp[8], *xp[8], *wsp, *xsp;
  const int piece = ((lane & 7) ^ mx_swizzle(lane >> 3)) * 16;
  auto begin_item = [&]() {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int row = 64 * wave + 8 * j + (lane >> 3);
      wp[j] = a.w + weight_row(row) * KB + piece;
      const int64_t src = token_row(row);
      xp[j] = (src < 0 ? zeros : a.x + src * KB) + piece;
    }
    const int64_t src = token_row(tid);
    wsp = a.w_mx + weight_row(tid) * SB;
    xsp = src < 0 ? zeros : a.x_mx + src * SB;
  };
  auto source = [&](const uint8_t* (&p)[8], int c, int j) {
    return 128 * c + piece < KB ? p[j] + 128 * c : zero;
  };
  auto load = [&](const uint8_t* from, uint8_t* buf, int j) {
    load_to_lds(from, buf + (64 * wave + 8 * j) * 128);
  };
  u32x4 sc[2];                                         // this thread's rows' scales of a round
  // (one load of 16 bytes, which needs no more than the dword's alignment: four of a dword each
  // are four requests for the line)
  // (loads from global memory in so many words: as flat ones they would not come back in order
  // with the loads into LDS, and those are counted)
  auto load_scales = [&](int r) {
    struct __attribute__((packed, aligned(4))) Piece { u32x4 v; };
    typedef const __attribute__((address_space(1))) Piece* PiecePtr;
    typedef const __attribute__((address_space(1))) uint32_t* WordPtr;
    if (16 * r + 16 <= SB) {
      sc[0] = ((PiecePtr)(wsp + 16 * r))->v;
      sc[1] = ((PiecePtr)(xsp + 16 * r))->v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int off = 16 * r + 4 * i;
        const bool in = off < SB;
        const uint32_t w = *(WordPtr)(wsp + (in ? off : 0)), x = *(WordPtr)(xsp + (in ? off : 0));
        sc[0][i] = in ? w : 0u;
        sc[1][i] = in ? x : 0u;
      }
    }
  };
  // dword g: bytes 2 g and 2 g + 1 of both chunks
  auto write_scales = [&]() {
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      const u32x4 v = sc[o];
      s_scale[kMxTile * o + tid] = u32x4{__builtin_amdgcn_perm(v[2], v[0], 0x05040100u),
                                         __builtin_amdgcn_perm(v[2], v[0], 0x07060302u),
                                         __builtin_amdgcn_perm(v[3], v[1], 0x05040100u),
                                         __builtin_amdgcn_perm(v[3], v[1], 0x07060302u)};
    }
  };
  // the loads' next round: the item's next, or the first of the next item (of this one again
  // behind the last item, so that the number of loads under way stays the same)
  auto advance = [&]() {
    if (++ld_r == nr) {
      ld_r = 0;
      more = walk.next(&ld, &ld_cb);
      if (more) begin_item();
    }
  };

  // One item whose rows fit 32 MG tokens; a wave has 16 MG of them.
  auto item = [&](auto mg_c) {
    constexpr int MG = decltype(mg_c)::value;
    const int t0 = 16 * MG * wm;
    const TileRows tr = ld;
    const int cb = ld_cb;
    f32x4 acc[8][MG];
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int m = 0; m < MG; ++m) acc[r][m] = f32x4{0, 0, 0, 0};
    // Products go in batches of two token groups (one with a single group).  A batch's fragments
    // are read during the batch before it: the compiler waits for all LDS reads under way wherever
    // it waits for one (loads into LDS count among them), so each batch begins with that wait and
    // then reads ahead.  Reads and loads stand between the products, one after each, where they
    // cost nothing: a wavefront issues in order, and one has its SIMD to itself.  A chunk's last
    // batch is left for after the next barrier, where it covers the first reads from the new chunk.
    constexpr int BG = MG < 2 ? 1 : 2, NB = MG / BG;
    u32x4 wf[2][8], xf[2][BG];
    uint32_t ws[8], xs[MG], ws_next[8], xs_next[MG];
    // this lane's fragments of a chunk's two steps (blocks 2 g and 2 g + 1; the other row groups
    // at fixed distances) and its scales
    const int w_at = (128 * wn + l16) * 128, x_at = (t0 + l16) * 128;
    const int at[2] = {((2 * g) ^ mx_swizzle(l16)) << 4, ((2 * g + 1) ^ mx_swizzle(l16)) << 4};
    const uint32_t* ws_at = reinterpret_cast<const uint32_t*>(s_scale) + 4 * (128 * wn + l16) + g;
    const uint32_t* xs_at = reinterpret_cast<const uint32_t*>(s_scale) + 4 * (kMxTile + t0 + l16) + g;
    auto weights = [&](const uint8_t* buf, int f, int r) {
      return *reinterpret_cast<const u32x4*>(buf + w_at + at[f] + 2048 * r);
    };
    auto tokens = [&](const uint8_t* buf, int f, int m) {
      return *reinterpret_cast<const u32x4*>(buf + x_at + at[f] + 2048 * m);
    };
    auto arrive = [&](bool wait) {
      __builtin_amdgcn_sched_barrier(0);
      if (wait) __builtin_amdgcn_s_waitcnt(wait_vm_lds(kMxBufLoads));
      else __builtin_amdgcn_s_waitcnt(kWaitLds);
      asm volatile("s_barrier" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    };
    // batch q of a chunk (step q / NB), side(k) between its products k and k + 1
    auto products = [&](auto uc, auto qc, auto side) {
      constexpr int U = decltype(uc)::value, Q = decltype(qc)::value, m0 = Q % NB * BG;
      ready();
      for_ring<8 * BG>([&](auto kc) {
        constexpr int k = decltype(kc)::value, w = k & 7, i = k >> 3;
        mx_mma_in_place<U>(wf[Q / NB][w], xf[Q & 1][i], acc[w][m0 + i], ws[w], xs[m0 + i]);
        side(kc);
        __builtin_amdgcn_sched_barrier(0);
      });
    };
    auto nothing = [](auto) {};
    // the first chunk is in LDS, and the first round's scales (the caller has seen to it); the
    // batch left over from before is one of zeros
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      wf[0][w] = weights(s_w0, 0, w);
      wf[1][w] = u32x4{0u, 0u, 0u, 0u};
      ws[w] = 0u;
    }
#pragma unroll
    for (int i = 0; i < BG; ++i) xf[1][i] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int m = 0; m < MG; ++m) xs[m] = 0u;
    for (int r = 0; r < nr; ++r) {
      for_ring<4>([&](auto uc) {
        constexpr int U = decltype(uc)::value, F = U & 1;
        const uint8_t *w_next = U == 0 || U == 3 ? s_w0 : s_w1, *x_here = U < 2 ? s_x0 : s_x1;
        // what this step reads is in LDS, and what the loads of this step overwrite has been
        // read; after the barrier that holds for the workgroup
        // (all that an item's first two steps read was waited for before the stores of the one
        // before: those are not waited for until two steps are done)
        arrive(U >= 2 || r > 0);
        if constexpr (F == 0) {
#pragma unroll
          for (int i = 0; i < BG; ++i) xf[0][i] = tokens(x_here, 0, i);
        }
        if constexpr (U == 0) {
#pragma unroll
          for (int w = 0; w < 8; ++w) ws_next[w] = ws_at[64 * w];
#pragma unroll
          for (int m = 0; m < MG; ++m) xs_next[m] = xs_at[64 * m];
        } else if constexpr (U == 1) {
          advance();
          load_scales(ld_r);
        } else if constexpr (U == 3) {
          write_scales();
        }
        // load j of this step: its source, and the load
        auto from = [&](int j) {
          if constexpr (U == 0) return source(xp, 2 * ld_r + 1, j);
          else if constexpr (U == 1) return source(wp, 2 * ld_r, j);
          else if constexpr (U == 2) return source(xp, 2 * ld_r, j);
          else return source(wp, 2 * ld_r + 1, j);
        };
        uint8_t* to = U == 0 ? s_x1 : U == 1 ? s_w0 : U == 2 ? s_x0 : s_w1;
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (F == 0) products(IntC<(U + 3) & 3>{}, IntC<2 * NB - 1>{}, nothing);
        if constexpr (U == 0) {
#pragma unroll
          for (int w = 0; w < 8; ++w) ws[w] = ws_next[w];
#pragma unroll
          for (int m = 0; m < MG; ++m) xs[m] = xs_next[m];
        }
        constexpr int kBatches = F == 0 ? NB : NB - 1;
        if constexpr (kBatches > 0) {
          for_ring<kBatches>([&](auto bc) {
            constexpr int B = decltype(bc)::value, Q = F * NB + B;
            constexpr int w0 = 8 * B / kBatches, nw = 8 * (B + 1) / kBatches - w0;
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(kWaitLds);
            const uint8_t* src = nullptr;
            // behind product k: the next batch's token rows, the next step's weights, and this
            // batch's share of the loads, each with its source one product earlier
            products(uc, IntC<Q>{}, [&](auto kc) {
              constexpr int k = decltype(kc)::value, last = 8 * BG - 1;
              auto side = [&](int i) {
                if (i < BG) {
                  xf[(Q + 1) & 1][i] = tokens(x_here, (Q + 1) / NB, (Q + 1) % NB * BG + i);
                } else if (i < BG + nw) {
                  wf[F ^ 1][w0 + i - BG] = weights(w_next, F ^ 1, w0 + i - BG);
                } else if (i < BG + nw + 2 * nw) {
                  const int j = (i - BG - nw) / 2;
                  if ((i - BG - nw) % 2 == 0) src = from(w0 + j);
                  else load(src, to, w0 + j);
                }
              };
              side(k);
              if constexpr (k == last) {
#pragma unroll
                for (int i = last + 1; i < BG + 3 * nw; ++i) side(i);
              }
            });
          });
        } else {
#pragma unroll
          for (int w = 0; w < 8; ++w) wf[0][w] = weights(w_next, 0, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) load(from(j), to, j);
        }
      });
      settle();
    }
    // the batch left over, by the builtin: its results are read next, and those waits the compiler
    // knows
#pragma unroll
    for (int i = 0; i < BG; ++i)
#pragma unroll
      for (int w = 0; w < 8; ++w)
        acc[w][MG - BG + i] = mx_mma<3>(wf[1][w], xf[1][i], acc[w][MG - BG + i], ws[w], xs[MG - BG + i]);
    __builtin_amdgcn_s_waitcnt(wait_vm_lds(0));
    const float beta = SITU ? uniform(a.beta ? a.beta[tr.expert] : 4.0f) : 0.0f;
    const float lam = SITU ? uniform(a.lam ? a.lam[tr.expert] : 25.0f) : 0.0f;
    const float ib = SITU ? uniform(1.0f / beta) : 0.0f, il = SITU ? uniform(1.0f / lam) : 0.0f;
    // eight consecutive columns of token group m
    auto columns = [&](int s, int m) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (SITU) {
          const int r = 4 * s + (i & 4) / 2;
          v[i] = situ_f32(acc[r][m][i & 3], acc[r + 1][m][i & 3], beta, ib, lam, il);
        } else {
          v[i] = acc[2 * s + (i >> 2)][m][i & 3];
        }
      }
      return u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                   pack_bf16x2(v[6], v[7])};
    };
    constexpr int kSpans = SITU ? 2 : 4;               // of 32 columns, eight per lane
    const int n0 = cb * kCols + kCols / 2 * wn + 8 * g, rows = tr.nrows - t0 - l16;
    uint16_t* o = a.out + static_cast<int64_t>(tr.row0 + t0 + l16) * a.N + n0;
    if (a.N % 8 == 0 && cb * kCols + kCols <= a.N) {
#pragma unroll
      for (int m = 0; m < MG; ++m) {
        if (16 * m < rows) {
#pragma unroll
          for (int s = 0; s < kSpans; ++s) *reinterpret_cast<u32x4*>(o + 32 * s) = columns(s, m);
        }
        o += static_cast<int64_t>(16) * a.N;
      }
    } else {
#pragma unroll
      for (int m = 0; m < MG; ++m) {
        if (16 * m < rows) {
#pragma unroll
          for (int s = 0; s < kSpans; ++s) store_columns(o + 32 * s, columns(s, m), a.N, n0 + 32 * s);
        }
        o += static_cast<int64_t>(16) * a.N;
      }
    }
  };

  begin_item();
  load_scales(0);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    load(source(wp, 0, j), s_w0, j);
    load(source(xp, 0, j), s_x0, j);
    load(source(wp, 1, j), s_w1, j);
  }
  write_scales();
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  do {
    if (ld.nrows > 128) item(IntC<8>{});
    else if (ld.nrows > 64) item(IntC<4>{});
    else if (ld.nrows > 32) item(IntC<2>{});
    else item(IntC<1>{});
  } while (more);
  __builtin_amdgcn_s_waitcnt(0);                       // no load into LDS outlives the workgroup
}

template <bool SITU>
static hipError_t launch_mx_big(const MxGroupedArgs& a, hipStream_t stream) {
  const unsigned grid = static_cast<unsigned>(a.cus / a.xcds * a.xcds);
  grouped_mx_big_kernel<SITU><<<dim3(grid), dim3(kMxThreads),
                                (static_cast<size_t>(a.E) + 1) * 8, stream>>>(a);
  return hipGetLastError();
}

template <bool SITU>
static hipError_t launch_mx_one(const MxGroupedArgs& a, hipStream_t stream) {
  const int64_t R = a.R, E = a.E, few = a.cus * 3 / 4;
  auto items = [&](int tile, int block) {
    return (std::min(R, E) + R / tile) * ((a.Nw + block - 1) / block);
  };
  if (E <= 1024 && R >= 448 * E && items(256, 256) >= few) return launch_mx_big<SITU>(a, stream);
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
