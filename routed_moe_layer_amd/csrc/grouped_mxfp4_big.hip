// The largest tiles of the products grouped by expert of microscaled FP4 rows (the mathematics and
// the operands' order in K: grouped_mxfp4.hip).
#include "common.h"
#include "grouped_mxfp4.h"
#include "kernels.h"

namespace rmoe {

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
// Before a batch of them whose operands vector instructions may have written, two wait states.
// (Inside a batch only LDS reads write operands, which are waited for.  An s_nop in front of each
// instruction took 4% of 8192^3.)
__device__ __forceinline__ void ready() { asm volatile("s_nop 1" ::: "memory"); }
// Behind the last of them in a loop, before its branch: on gfx950 a 4-pass instruction's result is
// there after eight wait states, and code behind the loop may read it at once.  s_nop 7 is exactly
// those eight, as the compiler puts behind the builtin; there is none to spare.
__device__ __forceinline__ void settle() { asm volatile("s_nop 7" ::: "memory"); }

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
// takes 251 to 256 us, 4.3 to 4.4 PFLOP/s (the instruction alone on random codes 6.7, with the clock
// down to 1.6 GHz; an earlier state at 4.0 made 4.6 without its loads and 4.7 without its LDS reads; the
// library's product 2.9), the matrix units busy 53% of the cycles at 1.9 GHz.  8 experts x 4096 rows
// (N = 3584, K = 4096) take 265 us, 3.6 PFLOP/s, in seven to eight rounds of items, 270 gathered: at a
// change of item nine entries of row_idx are waited for one by one.  Where K is no multiple of 512 the
// last scales are, too: K = 4224, 3% more work, takes 302 us.  Eight wavefronts of 128 x 64 products
// read 1.5 times as much from LDS.
//
// With SiTU 33 registers spill (136 bytes a lane), and the activation is not covered by the next item's
// products: 8 experts x 4096 rows, N = 1792, K = 4096 take 365 us where the same products without it
// take 265; 32768 rows, N = 1024, K = 2048 145 and 94.
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
  mx_scan<kMxWaves>(a, s_tile, a.R / kMxTile, [](int n) { return n / kMxTile; });
  mx_scan<kMxWaves>(a, s_tile + a.E + 1, 2 * min(a.R, a.E), [](int n) {
    return (n % kMxTile + kMxTile / 2 - 1) / (kMxTile / 2);
  });
  constexpr int kCols = kMxTile / (SITU ? 2 : 1);
  const int nblk = (a.N + kCols - 1) / kCols;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int g = lane >> 4, l16 = lane & 15;
  const int wn = wave & 1, wm = wave >> 1;             // the wave's weight half and token half
  const int KB = a.KB, SB = a.SB;
  const int nr = (KB + 255) / 256;                     // rounds of two chunks
  const uint8_t* zeros = reinterpret_cast<const uint8_t*>(g_zero_row);
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
    return min(n, a.N - 1) + (SITU && (r & 1) ? a.N : 0);
  };
  // source row of token row i, -1 for zeros; rows that are not there read the first of the tile,
  // and the epilogue leaves them out
  auto token_row = [&](int i) { return source_row(a, ld.row0 + (i < ld.nrows ? i : 0)); };
  // Load j of a wave fills rows 64 wave + 8 j + lane / 8 of an operand, slot lane % 8 of a row
  // with piece (lane % 8) ^ mx_swizzle(row).  Thread t loads the scales of row t of both operands.
  // Offsets from the expert's first weights, and from all token rows or (nothing gathers them) the
  // tile's first.
  uint32_t wo[8], xo[8];
  buffer_t w_buf, x_buf;
  const uint8_t *wsp, *xsp;
  const int piece = ((lane & 7) ^ mx_swizzle(lane >> 3)) * 16;
  auto begin_item = [&]() __attribute__((always_inline)) {
    const int64_t w_at = static_cast<int64_t>(ld.expert) * a.Nw;
    const uint8_t* w = a.w + w_at * KB;
    const bool gathered = a.row_idx != nullptr;
    const int first = gathered ? 0 : __builtin_amdgcn_readfirstlane(ld.row0);
    const int rows = gathered ? a.x_rows : __builtin_amdgcn_readfirstlane(ld.nrows);
    w_buf = mx_buffer(w, static_cast<uint32_t>(a.Nw) * KB);
    x_buf = mx_buffer(a.x + static_cast<int64_t>(first) * KB, static_cast<uint32_t>(rows) * KB);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int row = 64 * wave + 8 * j + (lane >> 3);
      const int64_t src = token_row(row);
      wo[j] = static_cast<uint32_t>(weight_row(row)) * KB + piece;
      xo[j] = src < 0 ? kNowhere : static_cast<uint32_t>(static_cast<int>(src) - first) * KB + piece;
    }
    const int64_t src = token_row(tid);
    wsp = a.w_mx + (w_at + weight_row(tid)) * SB;
    xsp = src < 0 ? zeros : a.x_mx + src * SB;
  };
  // load j of chunk c of the weights or the token rows: where from (source), and the load
  auto source = [&](auto weights, int c, int j) {
    const bool in = 128 * c + piece < KB;
    return in ? (weights.value ? wo[j] : xo[j]) : kNowhere;
  };
  auto load = [&](auto weights, uint32_t from, int c, uint8_t* buf, int j) {
    mx_load<16>(weights.value ? w_buf : x_buf, from, 128 * c, buf + (64 * wave + 8 * j) * 128);
  };
  u32x4 sc[2];                                         // this thread's rows' scales of a round
  // (one load of 16 bytes, which needs no more than the dword's alignment: four of a dword each
  // are four requests for the line)
  // (loads from global memory in so many words: as flat ones they would not come back in order
  // with the loads into LDS, and those are counted)
  auto load_scales = [&](int r) __attribute__((always_inline)) {
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
  auto write_scales = [&]() __attribute__((always_inline)) {
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
  auto advance = [&]() __attribute__((always_inline)) {
    if (++ld_r == nr) {
      ld_r = 0;
      more = walk.next(&ld, &ld_cb);
      if (more) begin_item();
    }
  };

  // One item whose rows fit 32 MG tokens; a wave has 16 MG of them.
  auto item = [&](auto mg_c) __attribute__((always_inline)) {
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
    auto arrive = [&](bool wait) __attribute__((always_inline)) {
      __builtin_amdgcn_sched_barrier(0);
      if (wait) __builtin_amdgcn_s_waitcnt(wait_vm_lds(kMxBufLoads));
      else __builtin_amdgcn_s_waitcnt(kWaitLds);
      asm volatile("s_barrier" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    };
    // batch q of a chunk (step q / NB), side(k) between its products k and k + 1
    auto products = [&](auto uc, auto qc, auto side) __attribute__((always_inline)) {
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
        const IntC<U == 1 || U == 3> which;
        const int lc = 2 * ld_r + (U == 0 || U == 3);
        auto from = [&](int j) { return source(which, lc, j); };
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
            uint32_t src = 0;
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
                  else load(which, src, lc, to, w0 + j);
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
          for (int j = 0; j < 8; ++j) load(which, from(j), lc, to, j);
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
    auto columns = [&](int s, int m) __attribute__((always_inline)) {
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
    const bool whole = a.N % 8 == 0 && cb * kCols + kCols <= a.N;
    for_ring<MG>([&](auto mc) __attribute__((always_inline)) {
      constexpr int m = decltype(mc)::value;
      if (16 * m < rows) {
        for_ring<kSpans>([&](auto sc) __attribute__((always_inline)) {
          constexpr int s = decltype(sc)::value;
          const u32x4 v = columns(s, m);
          if (whole) *reinterpret_cast<u32x4*>(o + 32 * s) = v;
          else store_columns(o + 32 * s, v, a.N, n0 + 32 * s);
        });
      }
      o += static_cast<int64_t>(16) * a.N;
    });
  };

  begin_item();
  load_scales(0);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    load(IntC<1>{}, source(IntC<1>{}, 0, j), 0, s_w0, j);
    load(IntC<0>{}, source(IntC<0>{}, 0, j), 0, s_x0, j);
    load(IntC<1>{}, source(IntC<1>{}, 1, j), 1, s_w1, j);
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

hipError_t launch_grouped_mxfp4_big(const MxGroupedArgs& a, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.cus / a.xcds * a.xcds)), block(kMxThreads);
  const size_t lds = (static_cast<size_t>(a.E) + 1) * 8;
  if (a.situ) grouped_mx_big_kernel<true><<<grid, block, lds, stream>>>(a);
  else grouped_mx_big_kernel<false><<<grid, block, lds, stream>>>(a);
  return hipGetLastError();
}

}  // namespace rmoe
