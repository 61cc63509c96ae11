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

// Eight consecutive columns n .. n + 7 of a row at o, those below N.  Where N is no multiple of 8 a
// row's columns are aligned to four or to one of them.
__device__ __forceinline__ void store_columns(uint16_t* o, u32x4 v, int N, int n) {
  if (N % 8 == 0) {
    if (n < N) *reinterpret_cast<u32x4*>(o) = v;
  } else if (N % 4 == 0) {
    if (n < N) *reinterpret_cast<uint2*>(o) = make_uint2(v[0], v[1]);
    if (n + 4 < N) *reinterpret_cast<uint2*>(o + 4) = make_uint2(v[2], v[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (n + i < N) o[i] = static_cast<uint16_t>(v[i >> 1] >> (16 * (i & 1)));
  }
}
// The same for four columns.
__device__ __forceinline__ void store_columns(uint16_t* o, uint2 v, int N, int n) {
  if (N % 4 == 0) {
    if (n < N) *reinterpret_cast<uint2*>(o) = v;
  } else {
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) o[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
  }
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
// Before a batch of them whose operands vector instructions may have written, two wait states.
// (Inside a batch only LDS reads write operands, which are waited for.  An s_nop in front of each
// instruction took 4% of 8192^3.)
__device__ __forceinline__ void ready() { asm volatile("s_nop 1" ::: "memory"); }
// Behind the last of them in a loop, before its branch: a 4-pass instruction's result is there
// after 7 wait states, and code behind the loop may read it at once.
__device__ __forceinline__ void settle() { asm volatile("s_nop 7" ::: "memory"); }

// Where loads into LDS read an operand.  Loads through a buffer descriptor take a 32-bit offset
// per lane and one for all lanes, and give zeros for an offset past its end (kNowhere): a load is
// one instruction behind the one that says where in LDS, its lanes' ends of K one more.  With
// addresses of 64 bits (WIDE, for operands of 4 GB and more: a workgroup's weights are one
// expert's, and its token rows those of a tile where nothing gathers them) it is three or four more,
// and a chunk's loads were most of what a wavefront did.
typedef __amdgpu_buffer_rsrc_t buffer_t;
constexpr uint32_t kNowhere = 0xFFFF0000u, kBufferMost = kNowhere;
__device__ __forceinline__ buffer_t mx_buffer(const uint8_t* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, static_cast<int>(bytes),
                                           0x00020000);
}
template <int BYTES>
__device__ __forceinline__ void mx_load(buffer_t from, uint32_t lane_off, int off, uint8_t* to) {
  if constexpr (BYTES == 16)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_ptr)to, 16, static_cast<int>(lane_off), off, 0, 0);
  else
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_ptr)to, 4, static_cast<int>(lane_off), off, 0, 0);
}

// The last i with s[i] <= v, for rising s[0 .. n] with s[0] <= v < s[n], n <= 2^18: 64 entries at a
// time are looked at by the lanes, so that a search is two or three LDS reads long.
__device__ __forceinline__ int mx_last_at_most(const int32_t* s, int n, int v) {
  const int lane = threadIdx.x & 63;
  int lo = 0, step = n > 4096 ? 4096 : n > 64 ? 64 : 1;
  for (;;) {
    const int i = lo + lane * step;
    const uint64_t in = __ballot(i < n && s[i] <= v);  // a run of lanes from 0 on
    lo += (__popcll(in) - 1) * step;
    if (step == 1) return __builtin_amdgcn_readfirstlane(lo);
    step /= 64;
  }
}

// scan_experts with the prefix sums read eight at a time: a workgroup of one or two wavefronts
// takes several rounds of them, and the latency of each is part of a small call's time.
template <int NW, class F>
__device__ __forceinline__ void mx_scan(const GroupedArgs& a, int32_t* s, int32_t most, F count) {
  constexpr int kThreads = NW * 64, kBatch = 8;
  for (int base = 0; base < a.E; base += kThreads * kBatch) {
    int32_t end[kBatch], begin[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int e = base + i * kThreads + static_cast<int>(threadIdx.x);
      end[i] = e < a.E ? a.cumsum[e] : 0;
      begin[i] = e > 0 && e < a.E ? a.cumsum[e - 1] : 0;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int e = base + i * kThreads + static_cast<int>(threadIdx.x);
      const int lo = min(max(begin[i], 0), a.R), hi = min(max(end[i], lo), a.R);
      if (e < a.E) s[e] = count(hi - lo);
    }
  }
  __syncthreads();
  __shared__ int32_t s_wave[NW];
  const int per = (a.E + kThreads - 1) / kThreads;
  const int lo = min(static_cast<int>(threadIdx.x) * per, a.E), hi = min(lo + per, a.E);
  int sum = 0;
  for (int e = lo; e < hi; ++e) sum += s[e];
  sum = min(sum, most);                  // (a cut part alone brings every later sum to the cut)
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
    const int n = s[e];
    s[e] = min(before, most);
    before += n;
  }
  if (threadIdx.x == kThreads - 1) s[a.E] = min(before, most);
  __syncthreads();
}

// Rows of expert e, the same for the whole wavefront, as expert_rows.  They come by scalar loads:
// a wait for vector ones would be one for all the loads under way.
__device__ __forceinline__ int2 mx_expert_rows(const GroupedArgs& a, int e) {
  typedef const __attribute__((address_space(4))) int32_t* ScalarPtr;
  const ScalarPtr cumsum = (ScalarPtr)a.cumsum;
  const int lo = e > 0 ? min(max(cumsum[e - 1], 0), a.R) : 0;
  return make_int2(lo, min(max(cumsum[e], lo), a.R));
}

// The source row of an entry of row_idx, or -1, as source_row.
__device__ __forceinline__ int64_t source_of(const GroupedArgs& a, int s) {
  if (s < 0) return -1;
  if (a.row_div > 1) s = static_cast<int>(static_cast<uint32_t>(s) / static_cast<uint32_t>(a.row_div));
  return s < a.x_rows ? s : -1;
}

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
// go from memory straight into LDS in chunks of 128 bytes of K, in a ring of S chunks that runs on
// over the borders between items: the load side is S - 1 chunks ahead of the products, with items
// of its own.  Every wavefront issues the same number of loads per chunk (the token rows' scales
// are loaded by several wavefronts alike), so one counted wait per chunk is enough: a chunk is
// there when no more loads are under way than were issued after it (stores behind them only make
// it wait for more).
//
// Bound by the bytes: FC1 of 16 tokens over 896 experts (N = 384 with SiTU, K = 3584, 328 MB) 71
// us, 4.6 TB/s; FC1 of 4096 tokens (1.37 GB) 331 us, 4.1 TB/s; FC2 of 1024 Zipf tokens (N = 3584,
// K = 384, 763 MB) 207 us, 3.7 TB/s, two chunks an item, half of the second of them zeros; a large
// read on the same card 5.99 TB/s.  A CU takes in about 20 bytes a ns this way, whether they come
// from memory or from a cache, and the token rows' count with the weights'.  Eight wavefronts per
// CU are needed for that: longer rings with four took 76 to 101 us for the 71.
// ---------------------------------------------------------------------------------------
//
// DIRECT: the source rows of a tile are read from row_idx, which the wavefront has to wait for
// with the loads around them.  Otherwise they are the sorted rows themselves or, of at most
// kMxListRows, in a list in LDS.
constexpr int kMxListRows = 2048;

template <bool SITU, bool DIRECT, bool WIDE, int BM, int NW, int PER_CU, int S>
__global__ __launch_bounds__(NW * 64, (NW * PER_CU + 3) / 4) void grouped_mx_mid_kernel(MxGroupedArgs a) {
  constexpr int kRows = 32 * NW, kCols = kRows / (SITU ? 2 : 1), MT = BM / 16;
  constexpr int kXLoads = BM / (8 * NW), kLoads = 6 + kXLoads;       // per wavefront and chunk
  constexpr int kXScaleLoads = BM < 32 ? 1 : BM / 32;                // of 32 rows
  static_assert(kXLoads * 8 * NW == BM && kXScaleLoads <= NW, "");
  // a buffer: weights, token rows, the weights' scales, the token rows' scales
  constexpr int kScales = (kRows + BM) * 128, kBytes = kScales + (kRows + 32 * kXScaleLoads) * 8;
  extern __shared__ int32_t s_tile[];
  __shared__ alignas(16) uint8_t s_0[kBytes], s_1[kBytes], s_2[kBytes];
  auto ring = [&](auto u) {
    constexpr int U = decltype(u)::value % S;
    if constexpr (U == 0) return &s_0[0];
    else if constexpr (U == 1) return &s_1[0];
    else if constexpr (U == 2) return &s_2[0];
    else return more_ring<U, kBytes>();
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
    __builtin_amdgcn_s_waitcnt(wait_vm_lds((S - 2) * kLoads));
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
  for_ring<S - 1>([&](auto u) { load(ring(u)); });
  clear();
  // An item may end at any buffer of the ring.  The steps of a round are taken whatever happens in
  // it, behind the last item on chunks that nobody stores: with a step left out on some path the
  // compiler no longer knows how many loads are under way and waits for all of them.
  int c = 0;
  bool alive = true;
  while (alive) {
    for_ring<S>([&](auto u) __attribute__((always_inline)) {
      arrive();
      load(ring(IntC<decltype(u)::value + S - 1>{}));
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

static bool mx_wide(const MxGroupedArgs& a) {
  return static_cast<uint64_t>(a.Nw) * a.KB > kBufferMost ||
         (a.row_idx && static_cast<uint64_t>(a.x_rows) * a.KB > kBufferMost);
}

template <bool SITU, int BM, int NW, int PER_CU, int S>
static hipError_t launch_mx_mid(const MxGroupedArgs& a, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.cus / a.xcds * a.xcds * PER_CU)), block(NW * 64);
  // the list has to fit behind the ring too (160 KB, less what the scan takes)
  constexpr size_t kRing = S * ((32 * NW + BM) * 128 + (32 * NW + (BM < 32 ? 32 : BM)) * 8);
  const size_t starts = (static_cast<size_t>(a.E) + 1) * 4, list = a.row_idx ? size_t(a.R) * 4 : 0;
  const bool direct = a.row_idx && (a.R > kMxListRows || kRing + starts + list > 163840 - 128 || mx_wide(a));
  const size_t lds = starts + (direct ? 0 : list);
  if (mx_wide(a)) {
    if (direct) grouped_mx_mid_kernel<SITU, true, true, BM, NW, PER_CU, S><<<grid, block, lds, stream>>>(a);
    else grouped_mx_mid_kernel<SITU, false, true, BM, NW, PER_CU, S><<<grid, block, lds, stream>>>(a);
  } else if (direct) {
    grouped_mx_mid_kernel<SITU, true, false, BM, NW, PER_CU, S><<<grid, block, lds, stream>>>(a);
  } else {
    grouped_mx_mid_kernel<SITU, false, false, BM, NW, PER_CU, S><<<grid, block, lds, stream>>>(a);
  }
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
// takes 241 us, 4.6 PFLOP/s (the instruction alone on random codes 6.7, with the clock down to
// 1.6 GHz; an earlier state at 4.0 made 4.6 without its loads and 4.7 without its LDS reads; the
// library's product 2.9).  8 experts x 4096 rows (N = 3584, K = 4096) take 267 us, 3.6 PFLOP/s, in
// seven to eight rounds of items.  Eight wavefronts of 128 x 64 products read 1.5 times as much from LDS.
// ---------------------------------------------------------------------------------------
constexpr int kWaitLds = 0xC07F;                       // s_waitcnt for LDS reads alone
constexpr int kMxTile = 256, kMxWaves = 4, kMxThreads = kMxWaves * 64;
constexpr int kMxBufBytes = kMxTile * 128, kMxBufLoads = kMxBufBytes / 1024 / kMxWaves;

template <bool SITU, bool WIDE>
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
    return min(n, a.N - 1) + (SITU && (r & 1) ? a.N : 0);
  };
  // source row of token row i, -1 for zeros; rows that are not there read the first of the tile,
  // and the epilogue leaves them out
  auto token_row = [&](int i) { return source_row(a, ld.row0 + (i < ld.nrows ? i : 0)); };
  // Load j of a wave fills rows 64 wave + 8 j + lane / 8 of an operand, slot lane % 8 of a row
  // with piece (lane % 8) ^ mx_swizzle(row).  Thread t loads the scales of row t of both operands.
  // Offsets (WIDE: addresses) as in the kernel above.
  uint32_t wo[8], xo[8];
  buffer_t w_buf, x_buf;
  const uint8_t *wp[8], *xp[8], *wsp, *xsp;
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
      if constexpr (WIDE) {
        wp[j] = w + static_cast<int64_t>(weight_row(row)) * KB + piece;
        xp[j] = (src < 0 ? zeros : a.x + src * KB) + piece;
      } else {
        wo[j] = static_cast<uint32_t>(weight_row(row)) * KB + piece;
        xo[j] = src < 0 ? kNowhere : static_cast<uint32_t>(static_cast<int>(src) - first) * KB + piece;
      }
    }
    const int64_t src = token_row(tid);
    wsp = a.w_mx + (w_at + weight_row(tid)) * SB;
    xsp = src < 0 ? zeros : a.x_mx + src * SB;
  };
  // load j of chunk c of the weights or the token rows: where from (source), and the load
  auto source = [&](auto weights, int c, int j) {
    const bool in = 128 * c + piece < KB;
    if constexpr (WIDE) return in ? (weights.value ? wp[j] : xp[j]) + 128 * c : zero;
    else return in ? (weights.value ? wo[j] : xo[j]) : kNowhere;
  };
  auto load = [&](auto weights, auto from, int c, uint8_t* buf, int j) {
    uint8_t* to = buf + (64 * wave + 8 * j) * 128;
    if constexpr (WIDE) load_to_lds(from, to);
    else if constexpr (weights.value) mx_load<16>(w_buf, from, 128 * c, to);
    else mx_load<16>(x_buf, from, 128 * c, to);
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
            decltype(from(0)) src{};
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

template <bool SITU>
static hipError_t launch_mx_big(const MxGroupedArgs& a, hipStream_t stream) {
  const unsigned grid = static_cast<unsigned>(a.cus / a.xcds * a.xcds);
  const size_t lds = (static_cast<size_t>(a.E) + 1) * 8;
  if (mx_wide(a)) grouped_mx_big_kernel<SITU, true><<<dim3(grid), dim3(kMxThreads), lds, stream>>>(a);
  else grouped_mx_big_kernel<SITU, false><<<dim3(grid), dim3(kMxThreads), lds, stream>>>(a);
  return hipGetLastError();
}

// Which kernel.  Larger tiles read the weights for more rows at once; smaller ones and smaller
// blocks of weight rows make more work items.  items() is an upper bound of the items of a kernel
// (the host does not know the rows of each expert), `few` three quarters of the CUs.  Measured on
// one MI355X, us with tiles of 256 / 128 / 64 rows by 256 weight rows, 64 by 128, 32 by 64 and 16
// by 64:
//   many rows per expert: 64 experts x 512 rows, N = K = 2048  130 / 146 / 190 / 183 / 287 / 438;
//     x 256 rows (half of the experts above one tile)  80 / 84 / 103 / 100 / 157 / 230, but 896 x
//     292 rows, N = 384 with SiTU, K = 3584  986 / 872 / 1138 / 1373 / 2282 / 2614; 8 x 256 rows,
//     N = K = 4096, whose tiles of 256 are one round of the chip  43 / 55 / 58 / 52 / 76 / 109;
//   fewer: 896 x 73 rows, the same N and K  440 / 347 / 458 / 522 / 707 / 798; 18 rows, N = 3584,
//     K = 384, Zipf  345 / 216 / 210 / 284 / 321 / 251; 4.6 rows  288 / 202 / 186 / 240 / 237 / 158;
//     1.1 rows, N = 384 with SiTU, K = 3584  112 / 77 / 76 / 85 / 83 / 72;
//   few items: 8 experts x 32 rows, N = K = 4096  26 / 24 / 24 / 18 / 24 / 28; one expert, N = K =
//     7168, 512 rows  52 / 46 / 36 / 36 / 52 / 81, 64 rows  34 / 34 / 33 / 21 / 15 / 17, 16 rows
//     33 / 29 / 28 / 18 / 13 / 13.
template <bool SITU>
static hipError_t launch_mx_one(const MxGroupedArgs& a, hipStream_t stream) {
  const int64_t R = a.R, E = a.E, some = std::min(R, E), few = a.cus * 3 / 4;
  auto items = [&](int tile, int block) { return (some + R / tile) * ((a.Nw + block - 1) / block); };
  // (the LDS of the larger tiles leaves room for so many experts' prefix sums)
  const int64_t items256 = items(256, 256);
  if (E <= 1024 && items256 >= few && (R >= 448 * E || (R >= 224 * E && items256 <= a.cus)))
    return launch_mx_big<SITU>(a, stream);
  if (items(128, 256) >= few) {
    if (E <= 1536 && R > 32 * E) return launch_mx_mid<SITU, 128, 8, 1, 3>(a, stream);
    if (E <= 8192 && R > 8 * E) return launch_mx_mid<SITU, 64, 8, 1, 3>(a, stream);
    if (R > 8 * E) return launch_mx_mid<SITU, 64, 4, 2, 3>(a, stream);
  } else if (R > 16 * some) {
    if (items(64, 128) >= few) return launch_mx_mid<SITU, 64, 4, 2, 3>(a, stream);
    return launch_mx_mid<SITU, 32, 2, 4, 3>(a, stream);
  }
  return launch_mx_mid<SITU, 16, 2, 4, 3>(a, stream);
}

hipError_t launch_grouped_mxfp4(const MxGroupedArgs& a, hipStream_t stream) {
  return a.situ ? launch_mx_one<true>(a, stream) : launch_mx_one<false>(a, stream);
}

}  // namespace rmoe
