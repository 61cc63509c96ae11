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
#include "common.h"
#include "grouped_mxfp4.h"
#include "grouped_mxfp4_rule.h"
#include "kernels.h"

namespace rmoe {

// The work items of a persistent workgroup, a tile and one block of weight rows each, in the order
// of ItemWalk: runs of kTileRun tiles, inside a run by weight block, inside a block by tile, runs
// dealt to the XCDs in turn or in equal contiguous parts.  There are fewer than 2^31 (at most 2^17 +
// 1536 tiles x 512 blocks, 2^18 + 10240 x 1024 or, of the smallest tiles, which few rows take,
// 2^15 x 2048), and a step is made without a division.
struct MxItemWalk {
  int tiles, nblk, xcd, step, run, rem, left;
  bool deal;
  __device__ __forceinline__ MxItemWalk(const GroupedArgs& a, int all_tiles, int blocks)
      : tiles(all_tiles), nblk(blocks) {
    xcd = static_cast<int>(blockIdx.x) % a.xcds;
    step = static_cast<int>(gridDim.x) / a.xcds;
    const int first = static_cast<int>(blockIdx.x) / a.xcds, per_run = kTileRun * nblk;
    const int runs = (tiles + kTileRun - 1) / kTileRun;
    deal = runs >= kDealRuns * a.xcds;
    int at = first;
    if (deal) {
      left = (runs - xcd + a.xcds - 1) / a.xcds * per_run - first;
    } else {
      const int64_t total = static_cast<int64_t>(tiles) * nblk;
      const int begin = static_cast<int>(total * xcd / a.xcds);
      left = static_cast<int>(total * (xcd + 1) / a.xcds) - begin - first;
      at += begin;
    }
    run = at / per_run;
    rem = at - run * per_run;
  }
  // The next item: its tile and weight block; false when there is none left.
  __device__ __forceinline__ bool next(int xcds, int* tile, int* cb) {
    const int per_run = kTileRun * nblk;
    while (left > 0) {
      const int r = deal ? run * xcds + xcd : run, m = rem;
      left -= step;
      rem += step;
      while (rem >= per_run) {
        rem -= per_run;
        ++run;
      }
      const int in_run = min(kTileRun, tiles - r * kTileRun);
      if (m >= in_run * nblk) continue;                // the last run may be short
      *cb = in_run == kTileRun ? m / kTileRun : m / in_run;
      *tile = r * kTileRun + (m - *cb * in_run);
      return true;
    }
    return false;
  }
};

// ---------------------------------------------------------------------------------------
// Tiles of up to BM rows (16, 32, 64 or 128).  A workgroup of NW wavefronts multiplies one tile of
// an expert's rows with 32 NW weight rows, 32 per wavefront.  Codes and scales of both operands
// go from memory straight into LDS in chunks of 128 bytes of K, in a ring of three that runs on
// over the borders between items: the load side is two chunks ahead of the products, with items
// of its own.  Every wavefront issues the same number of loads per chunk (the token rows' scales
// are loaded by several wavefronts alike), so one counted wait per chunk is enough: a chunk is
// there when no more loads are under way than were issued after it (stores behind them only make
// it wait for more).
//
// Bound by the bytes: FC1 of 16 tokens over 896 experts (N = 384 with SiTU, K = 3584, 328 MB) 71
// us, 4.6 TB/s; FC1 of 4096 tokens (1.37 GB) 331 us, 4.1 TB/s; FC2 of 1024 Zipf tokens (N = 3584,
// K = 384, 763 MB) 209 us, 3.6 TB/s, two chunks an item, half of the second of them zeros; a large
// read on the same card 5.99 TB/s.  A CU takes in 17 to 24 bytes a ns this way, however many of
// them the L2 holds (of the three's requests 63, 44 and 53% miss it), and the token rows' count with the
// weights'.  Eight wavefronts per
// CU are needed for that: longer rings with four took 76 to 101 us for the 71.
// ---------------------------------------------------------------------------------------
//
// DIRECT: the source rows of a tile are read from row_idx, which the wavefront has to wait for
// with the loads around them.  Otherwise they are the sorted rows themselves or, of at most
// kMxListRows, in a list in LDS.

template <bool SITU, bool DIRECT, bool WIDE, int BM, int NW, int PER_CU>
__global__ __launch_bounds__(NW * 64, (NW * PER_CU + 3) / 4) void grouped_mx_mid_kernel(MxGroupedArgs a) {
  constexpr int kRows = 32 * NW, kCols = kRows / (SITU ? 2 : 1), MT = BM / 16;
  constexpr int kXLoads = BM / (8 * NW), kLoads = 6 + kXLoads;       // per wavefront and chunk
  constexpr int kXScaleLoads = BM < 32 ? 1 : BM / 32;                // of 32 rows
  static_assert(kXLoads * 8 * NW == BM && kXScaleLoads <= NW, "");
  // a buffer: weights, token rows, the weights' scales, the token rows' scales
  constexpr int kScales = (kRows + BM) * 128, kBytes = kScales + (kRows + 32 * kXScaleLoads) * 8;
  static_assert(kMxRing * kBytes == mx_ring_bytes(MxTiles{BM, NW, PER_CU, WIDE}), "");
  extern __shared__ int32_t s_tile[];
  __shared__ alignas(16) uint8_t s_0[kBytes], s_1[kBytes], s_2[kBytes];
  auto ring = [&](auto u) {
    constexpr int U = decltype(u)::value % kMxRing;
    return U == 0 ? &s_0[0] : U == 1 ? &s_1[0] : &s_2[0];
  };
  mx_scan<NW>(a, s_tile, a.R / BM + min(a.R, a.E), [](int n) { return (n + BM - 1) / BM; });
  const int nblk = (a.N + kCols - 1) / kCols;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int g = lane >> 4, l16 = lane & 15;
  const int KB = a.KB, SB = a.SB;
  const int nc = max((KB + 127) / 128, 2);             // (chunks past the end of K are zeros)
  int32_t* s_source = s_tile + a.E + 1;                // the list
  if (!DIRECT && a.row_idx) {
    for (int i = tid; i < a.R; i += NW * 64) s_source[i] = static_cast<int32_t>(source_row(a, i));
    __syncthreads();
  }
  const uint8_t *zero = reinterpret_cast<const uint8_t*>(&g_zero16),
                *zeros = reinterpret_cast<const uint8_t*>(g_zero_row);

  // An expert's rows are dealt evenly to its tiles in multiples of 16 (find_tile_even); the last
  // tiles of an expert may hold no row.
  struct Item {
    int expert, row0, nrows, cb;
  };
  auto next_item = [&](MxItemWalk& walk, Item* it) __attribute__((always_inline)) {
    int tile;
    while (walk.next(a.xcds, &tile, &it->cb)) {
      const int e = mx_last_at_most(s_tile, a.E, tile);
      const int2 r = mx_expert_rows(a, e);
      const int cnt = r.y - r.x, nt = (cnt + BM - 1) / BM;
      const int per = nt == 1 ? BM : ((cnt + nt - 1) / nt + 15) / 16 * 16;
      it->expert = e;
      it->row0 = __builtin_amdgcn_readfirstlane(r.x + (tile - s_tile[e]) * per);
      it->nrows = min(per, r.y - it->row0);
      if (it->nrows > 0) return true;
    }
    return false;
  };
  MxItemWalk load_walk(a, s_tile[a.E], nblk), walk = load_walk;
  Item ld, it;
  if (!next_item(walk, &it)) return;                   // the whole workgroup

  // Load j of a wavefront fills rows 8 j + lane / 8 of its 32 weight rows, or of its token rows,
  // slot lane % 8 of a row with piece (lane % 8) ^ mx_swizzle(row).  A load of scales takes 32
  // rows, two lanes each.
  // Offsets from the expert's first weights, and from all token rows or (nothing gathers them) the
  // tile's first; WIDE: addresses.
  uint32_t wo[4], wso, xo[kXLoads], xso;
  buffer_t w_buf, ws_buf, x_buf, xs_buf;
  const uint8_t *wp[4], *wsp, *xp[kXLoads], *xsp;
  const int piece = ((lane & 7) ^ mx_swizzle(lane >> 3)) * 16, half = (lane & 1) * 4;
  const int xs_row = 32 * (wave % kXScaleLoads);
  // LDS row 16 r + m of a wavefront's weights holds MFMA row m of group r: columns 8 (m / 4) +
  // 4 r + m % 4 of its 32, so that a lane's two groups make eight consecutive columns; with SiTU
  // column m, the gate row in group 0 and the up row in group 1
  auto weight_row = [&](int i) {
    const int r = i >> 4, m = i & 15;
    const int n = ld.cb * kCols + wave * (kCols / NW) + (SITU ? m : 8 * (m >> 2) + 4 * r + (m & 3));
    return static_cast<uint32_t>(min(n, a.N - 1) + (SITU && r ? a.N : 0));
  };
  // An item's first half is done a chunk before it begins: which one it is, and (DIRECT) the loads
  // of its row_idx, so that they are there by the second.
  Item next;
  bool more = true;
  int idx[kXLoads + 1];
  auto prepare = [&]() __attribute__((always_inline)) {
    more = next_item(load_walk, &next);
    if (!more || !DIRECT) return;
    // rows that are not there read the first of the tile, and the epilogue leaves them out
    auto row = [&](int i) { return a.row_idx[next.row0 + (i < next.nrows ? i : 0)]; };
#pragma unroll
    for (int j = 0; j < kXLoads; ++j) idx[j] = row(8 * (NW * j + wave) + (lane >> 3));
    idx[kXLoads] = row(xs_row + (lane >> 1));
  };
  auto begin_item = [&]() __attribute__((always_inline)) {
    if (!more) return;                                 // the last item again
    ld = next;
    const int64_t w_at = static_cast<int64_t>(ld.expert) * a.Nw;
    const uint8_t *w = a.w + w_at * KB, *ws = a.w_mx + w_at * SB;
    auto source = [&](int i, int j) -> int64_t {
      if constexpr (DIRECT) return source_of(a, idx[j]);
      const int row = ld.row0 + (i < ld.nrows ? i : 0);
      return a.row_idx ? s_source[row] : row;
    };
    if constexpr (WIDE) {
#pragma unroll
      for (int j = 0; j < 4; ++j) wp[j] = w + static_cast<int64_t>(weight_row(8 * j + (lane >> 3))) * KB + piece;
      wsp = ws + static_cast<int64_t>(weight_row(lane >> 1)) * SB + half;
#pragma unroll
      for (int j = 0; j < kXLoads; ++j) {
        const int64_t src = source(8 * (NW * j + wave) + (lane >> 3), j);
        xp[j] = (src < 0 ? zeros : a.x + src * KB) + piece;
      }
      const int64_t src = source(xs_row + (lane >> 1), kXLoads);
      xsp = (src < 0 ? zeros : a.x_mx + src * SB) + half;
    } else {
      w_buf = mx_buffer(w, static_cast<uint32_t>(a.Nw) * KB);
      ws_buf = mx_buffer(ws, static_cast<uint32_t>(a.Nw) * SB);
#pragma unroll
      for (int j = 0; j < 4; ++j) wo[j] = weight_row(8 * j + (lane >> 3)) * KB + piece;
      wso = weight_row(lane >> 1) * SB + half;
      const bool gathered = a.row_idx != nullptr;
      const int first = gathered ? 0 : ld.row0, rows = gathered ? a.x_rows : ld.nrows;
      x_buf = mx_buffer(a.x + static_cast<int64_t>(first) * KB, static_cast<uint32_t>(rows) * KB);
      xs_buf = mx_buffer(a.x_mx + static_cast<int64_t>(first) * SB, static_cast<uint32_t>(rows) * SB);
#pragma unroll
      for (int j = 0; j < kXLoads; ++j) {
        const int src = static_cast<int>(source(8 * (NW * j + wave) + (lane >> 3), j));
        xo[j] = src < 0 ? kNowhere : static_cast<uint32_t>(src - first) * KB + piece;
      }
      const int src = static_cast<int>(source(xs_row + (lane >> 1), kXLoads));
      xso = src < 0 ? kNowhere : static_cast<uint32_t>(src - first) * SB + half;
    }
  };
  // The load side's next chunk.  Behind the last item it loads that one again, so that the number
  // of loads under way stays the same.
  int lc = 0;
  auto load = [&](uint8_t* buf) __attribute__((always_inline)) {
    if (lc + 2 == nc) prepare();
    const int off = 128 * lc, soff = 8 * lc;
    const bool in = off + piece < KB, s_in = soff + half < SB;
    auto to = [&](int j) { return buf + (32 * wave + 8 * j) * 128; };
    auto x_to = [&](int j) { return buf + (kRows + 8 * (NW * j + wave)) * 128; };
    uint8_t *ws_to = buf + kScales + 32 * wave * 8, *xs_to = buf + kScales + (kRows + xs_row) * 8;
    if constexpr (WIDE) {
#pragma unroll
      for (int j = 0; j < 4; ++j) load_to_lds(in ? wp[j] + off : zero, to(j));
#pragma unroll
      for (int j = 0; j < kXLoads; ++j) load_to_lds(in ? xp[j] + off : zero, x_to(j));
      load4_to_lds(s_in ? wsp + soff : zero, ws_to);
      load4_to_lds(s_in ? xsp + soff : zero, xs_to);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) mx_load<16>(w_buf, in ? wo[j] : kNowhere, off, to(j));
#pragma unroll
      for (int j = 0; j < kXLoads; ++j) mx_load<16>(x_buf, in ? xo[j] : kNowhere, off, x_to(j));
      mx_load<4>(ws_buf, s_in ? wso : kNowhere, soff, ws_to);
      mx_load<4>(xs_buf, s_in ? xso : kNowhere, soff, xs_to);
    }
    if (++lc == nc) {
      lc = 0;
      begin_item();
    }
  };
  // this wavefront's loads of the chunk are in LDS, and it is done reading the buffers that the
  // next loads write; after the barrier that holds for the workgroup
  auto arrive = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(wait_vm_lds((kMxRing - 2) * kLoads));
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };

  f32x4 acc[2][MT];
  auto clear = [&]() {
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[r][m] = f32x4{0, 0, 0, 0};
  };
  auto compute = [&](const uint8_t* buf) __attribute__((always_inline)) {
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
      if (m == 0 || 16 * m < it.nrows) {
        const int row = kRows + 16 * m + l16;
        const u32x4 x0 = fragment(row, 0), x1 = fragment(row, 1);
        const uint32_t xs = scales(row);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          acc[r][m] = mx_mma<0>(wf[r][0], x0, acc[r][m], ws[r], xs);
          acc[r][m] = mx_mma<1>(wf[r][1], x1, acc[r][m], ws[r], xs);
        }
        // (read all at once the fragments of eight groups spilled)
        if constexpr (MT > 4) {
          if (m % 2 == 1) __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  };
  auto epilogue = [&]() __attribute__((always_inline)) {
    const int n = it.cb * kCols + wave * (kCols / NW) + (SITU ? 4 * g : 8 * g);
    float beta = 0, ib = 0, lam = 0, il = 0;
    if constexpr (SITU) {
      beta = uniform(a.beta ? a.beta[it.expert] : 4.0f);
      lam = uniform(a.lam ? a.lam[it.expert] : 25.0f);
      ib = uniform(1.0f / beta);
      il = uniform(1.0f / lam);
    }
    uint16_t* o = a.out + static_cast<int64_t>(it.row0 + l16) * a.N + n;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (16 * m + l16 < it.nrows) {
        if constexpr (SITU) {
          float v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = situ_f32(acc[0][m][i], acc[1][m][i], beta, ib, lam, il);
          store_columns(o, make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])), a.N, n);
        } else {
          const f32x4 c = acc[0][m], d = acc[1][m];
          store_columns(o, u32x4{pack_bf16x2(c[0], c[1]), pack_bf16x2(c[2], c[3]),
                                 pack_bf16x2(d[0], d[1]), pack_bf16x2(d[2], d[3])}, a.N, n);
        }
      }
      o += static_cast<int64_t>(16) * a.N;
    }
  };

  prepare();
  begin_item();
  for_ring<kMxRing - 1>([&](auto u) { load(ring(u)); });
  clear();
  // An item may end at any buffer of the ring.  The steps of a round are taken whatever happens in
  // it, behind the last item on chunks that nobody stores: with a step left out on some path the
  // compiler no longer knows how many loads are under way and waits for all of them.
  int c = 0;
  bool alive = true;
  while (alive) {
    for_ring<kMxRing>([&](auto u) __attribute__((always_inline)) {
      arrive();
      load(ring(IntC<decltype(u)::value + kMxRing - 1>{}));
      compute(ring(u));
      if (++c == nc) {
        c = 0;
        if (alive) {
          epilogue();
          clear();
          alive = next_item(walk, &it);
        }
      }
    });
  }
  __builtin_amdgcn_s_waitcnt(0);                       // no load into LDS outlives the workgroup
}

template <bool SITU, bool WIDE, int BM, int NW, int PER_CU>
static hipError_t launch_mx_mid(const MxGroupedArgs& a, const MxSizes& s, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.cus / a.xcds * a.xcds * PER_CU)), block(NW * 64);
  const bool direct = mx_direct(s, MxTiles{BM, NW, PER_CU, WIDE});
  const size_t list = a.row_idx && !direct ? size_t(a.R) * 4 : 0;
  const size_t lds = (static_cast<size_t>(a.E) + 1) * 4 + list;
  if (direct) grouped_mx_mid_kernel<SITU, true, WIDE, BM, NW, PER_CU><<<grid, block, lds, stream>>>(a);
  else grouped_mx_mid_kernel<SITU, false, WIDE, BM, NW, PER_CU><<<grid, block, lds, stream>>>(a);
  return hipGetLastError();
}

template <bool SITU>
static hipError_t launch_mx_one(const MxGroupedArgs& a, hipStream_t stream) {
  const MxSizes s{a.R, a.E, a.Nw, a.KB, a.x_rows, a.row_idx != nullptr, a.cus};
  const MxTiles t = mx_tiles(s);
  if (t.rows == 256) return launch_grouped_mxfp4_big(a, stream);
  if (t.rows == 128) return launch_mx_mid<SITU, false, 128, 8, 1>(a, s, stream);
  if (t.rows == 64 && t.waves == 8) return launch_mx_mid<SITU, false, 64, 8, 1>(a, s, stream);
  if (t.rows == 64 && t.wide) return launch_mx_mid<SITU, true, 64, 4, 2>(a, s, stream);
  if (t.rows == 64) return launch_mx_mid<SITU, false, 64, 4, 2>(a, s, stream);
  if (t.rows == 32) return launch_mx_mid<SITU, false, 32, 2, 4>(a, s, stream);
  if (t.wide) return launch_mx_mid<SITU, true, 16, 2, 4>(a, s, stream);
  return launch_mx_mid<SITU, false, 16, 2, 4>(a, s, stream);
}

hipError_t launch_grouped_mxfp4(const MxGroupedArgs& a, hipStream_t stream) {
  return a.situ ? launch_mx_one<true>(a, stream) : launch_mx_one<false>(a, stream);
}

}  // namespace rmoe
