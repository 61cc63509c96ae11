// Device helpers of the products grouped by expert (grouped.hip).
#pragma once

#include "common.h"
#include "kernels.h"

namespace rmoe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

template <int V>
struct IntC { static constexpr int value = V; };

// Operand types by their moe_quant_t value: 0 BF16, 1 int8, 3 E4M3.
template <int Q> struct AccOf { typedef f32x4 type; };
template <> struct AccOf<1> { typedef i32x4 type; };

// acc += A * B over one 128-byte chunk of K (two 16-byte fragments per lane and operand).
// Any order of K inside the chunk gives the same sum as long as both operands use it.
//
// BF16 products are added in fp32 and int8 products exactly in int32.  The E4M3 instructions
// (both the 32 and the 128 long one) first bring eight products to the exponent of the largest
// and cut bits below 2^-13 of it, then add in fp32; a product of two rounded E4M3 values is
// itself off by up to 2^-3.  Widening E4M3 to BF16 first would keep those bits at half the
// rate: 16x16x128 E4M3 takes the cycles of two 16x16x32 BF16.
template <int Q>
__device__ __forceinline__ typename AccOf<Q>::type mma_chunk(u32x4 a0, u32x4 a1, u32x4 b0,
                                                             u32x4 b1,
                                                             typename AccOf<Q>::type acc) {
  if constexpr (Q == 0) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a0),
                                                  __builtin_bit_cast(bf16x8, b0), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a1),
                                                  __builtin_bit_cast(bf16x8, b1), acc, 0, 0, 0);
  } else if constexpr (Q == 1) {
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a0),
                                                __builtin_bit_cast(i32x4, b0), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a1),
                                                __builtin_bit_cast(i32x4, b1), acc, 0, 0, 0);
  } else {
    i32x8 x, y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = static_cast<int>(a0[i]); x[4 + i] = static_cast<int>(a1[i]);
      y[i] = static_cast<int>(b0[i]); y[4 + i] = static_cast<int>(b1[i]);
    }
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc, 0, 0, 0, 0, 0, 0);   // unscaled
  }
  return acc;
}

// Rows of expert e, kept inside [0, R] whatever the prefix sums hold.
__device__ __forceinline__ int2 expert_rows(const GroupedArgs& a, int e) {
  const int lo = e > 0 ? min(max(a.cumsum[e - 1], 0), a.R) : 0;
  const int hi = min(max(a.cumsum[e], lo), a.R);
  return make_int2(lo, hi);
}

// s[e] = sum of count(rows of expert) over the experts before e, s[E] the total, all cut at
// `most`, the largest total of rising prefix sums.  (Falling ones give the same rows to several
// experts: uncut, 10240 experts that claim 2^24 rows in turn make 1.3e9 tiles of 64 rows times
// the blocks of weight rows, a launch that lasts for minutes.  Tiles past the cut are left out.)
// Every thread of the workgroup (NW wavefronts) calls this; it ends with a barrier.
template <int NW, class F>
__device__ __forceinline__ void scan_experts(const GroupedArgs& a, int32_t* s, int32_t most,
                                             F count) {
  __shared__ int32_t s_wave[NW];
  constexpr int kThreads = NW * 64;
  const int per = (a.E + kThreads - 1) / kThreads;
  const int lo = min(static_cast<int>(threadIdx.x) * per, a.E), hi = min(lo + per, a.E);
  int sum = 0;
  for (int e = lo; e < hi; ++e) {
    const int2 r = expert_rows(a, e);
    const int n = count(r.y - r.x);
    s[e] = n;
    sum += n;
  }
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

struct TileRows {
  int expert, row0, nrows;
};
// The expert of tile `tile`: the last one whose tiles start at or before it; s as from
// scan_experts, 0 <= tile < s[E].
__device__ __forceinline__ int tile_expert(const int32_t* s, int E, int tile) {
  int lo = 0, hi = E;                    // s[lo] <= tile < s[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s[mid] <= tile) lo = mid; else hi = mid;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// Tiles of up to BM rows with an expert's rows dealt evenly to them in multiples of 16 (so
// none is nearly empty while others are full); the last tiles of an expert may hold no row.
template <int BM>
__device__ __forceinline__ TileRows find_tile_even(const GroupedArgs& a, const int32_t* s_tile,
                                                   int tile) {
  const int e = tile_expert(s_tile, a.E, tile);
  const int2 r = expert_rows(a, e);
  const int cnt = r.y - r.x, nt = (cnt + BM - 1) / BM;
  const int per = ((cnt + nt - 1) / nt + 15) / 16 * 16;
  const int row0 = r.x + (tile - s_tile[e]) * per;
  return TileRows{e, row0, min(per, r.y - row0)};
}

// The work items of a persistent workgroup: an item is a tile and one block of weight rows.
// Items come in runs of kTileRun tiles (tiles of one expert read the same weights), inside a
// run by weight block, inside a block by tile.  An XCD works on whole runs, so an item's
// neighbours share its L2: with many runs they are dealt to the XCDs in turn (popular experts
// may lie next to each other), with few (below kDealRuns per XCD) each XCD takes an equal
// contiguous part of all items.  blockIdx.x counts XCDs first; gridDim.x is a multiple of
// their number.
constexpr int kTileRun = 4, kDealRuns = 8;
struct ItemWalk {
  const GroupedArgs& a;
  const int32_t* s_tile;
  int nblk, tiles, xcd, step;
  bool deal;
  int64_t at, end;
  __device__ __forceinline__ ItemWalk(const GroupedArgs& args, const int32_t* tile_starts, int blocks)
      : a(args), s_tile(tile_starts), nblk(blocks), tiles(tile_starts[args.E]) {
    xcd = static_cast<int>(blockIdx.x) % a.xcds;
    step = static_cast<int>(gridDim.x) / a.xcds;
    at = static_cast<int>(blockIdx.x) / a.xcds;
    const int runs = (tiles + kTileRun - 1) / kTileRun;
    deal = runs >= kDealRuns * a.xcds;
    if (deal) {
      end = static_cast<int64_t>((runs - xcd + a.xcds - 1) / a.xcds) * kTileRun * nblk;
    } else {
      const int64_t total = static_cast<int64_t>(tiles) * nblk;
      end = total * (xcd + 1) / a.xcds;
      at += total * xcd / a.xcds;
    }
  }
  // The next item with rows; false when there is none left.
  template <int BM>
  __device__ __forceinline__ bool next(TileRows* tr, int* cb) {
    const int per_run = kTileRun * nblk;               // N <= 65536: below 2^17
    while (at < end) {
      int run = static_cast<int>(at / per_run);
      const int rem = static_cast<int>(at - static_cast<int64_t>(run) * per_run);
      at += step;
      if (deal) run = run * a.xcds + xcd;
      const int in_run = min(kTileRun, tiles - run * kTileRun);
      if (rem >= in_run * nblk) continue;              // the last run may be short
      *cb = rem / in_run;
      *tr = find_tile_even<BM>(a, s_tile, run * kTileRun + rem % in_run);
      if (tr->nrows > 0) return true;
    }
    return false;
  }
};

// The same for tiles of BM rows that all cost the same, and up to two smaller ones (of up to
// half as many rows) per expert for the rest of its rows: the full tiles are dealt first, in
// equal contiguous parts to the XCDs and one by one to an XCD's workgroups, then the smaller
// ones, starting with the workgroups that got fewer of the full ones.
template <int BM>
struct FullFirstWalk {
  const GroupedArgs& a;
  const int32_t *s_full, *s_part;        // prefix sums of the full and the smaller tiles
  int nblk, step, slot, xcd;
  bool part = false;
  int64_t at, end;
  __device__ __forceinline__ FullFirstWalk(const GroupedArgs& args, const int32_t* full,
                                           const int32_t* smaller, int blocks)
      : a(args), s_full(full), s_part(smaller), nblk(blocks) {
    xcd = static_cast<int>(blockIdx.x) % a.xcds;
    step = static_cast<int>(gridDim.x) / a.xcds;
    slot = static_cast<int>(blockIdx.x) / a.xcds;
    range(s_full[a.E], slot);
  }
  __device__ __forceinline__ void range(int tiles, int first) {
    const int64_t total = static_cast<int64_t>(tiles) * nblk;
    at = total * xcd / a.xcds;
    end = total * (xcd + 1) / a.xcds;
    at += first;
  }
  __device__ __forceinline__ bool next(TileRows* tr, int* cb) {
    if (at >= end && !part) {
      part = true;
      // (at - end) % step: this workgroup's place behind those that the last round left out
      range(s_part[a.E], static_cast<int>((at - end) % step));
    }
    if (at >= end) return false;
    const int32_t* s = part ? s_part : s_full;
    const int per_run = kTileRun * nblk;
    const int run = static_cast<int>(at / per_run);
    const int rem = static_cast<int>(at - static_cast<int64_t>(run) * per_run);
    const int in_run = min(kTileRun, s[a.E] - run * kTileRun);
    const int tile = run * kTileRun + rem % in_run;
    at += step;
    *cb = rem / in_run;
    const int e = tile_expert(s, a.E, tile);
    const int2 r = expert_rows(a, e);
    const int row0 = part ? r.x + (r.y - r.x) / BM * BM + (tile - s[e]) * (BM / 2)
                          : r.x + (tile - s[e]) * BM;
    *tr = TileRows{e, row0, min(part ? BM / 2 : BM, r.y - row0)};
    return true;
  }
};

// Row of x that sorted row i reads, or -1 (zeros) when the index points outside x.
__device__ __forceinline__ int64_t source_row(const GroupedArgs& a, int i) {
  int s = i;
  if (a.row_idx) {
    s = a.row_idx[i];
    if (s < 0) return -1;
    if (a.row_div > 1) s = static_cast<int>(static_cast<uint32_t>(s) / static_cast<uint32_t>(a.row_div));
  }
  return s < a.x_rows ? s : -1;
}

// |tanh(v)| as a quotient num / den: an odd polynomial for |v| < 1/4 (next Taylor term below
// 2^-26 of the value), where 1 - exp(-2|v|) would cancel; else (1 - e) / (1 + e), e = exp(-2|v|).
__device__ __forceinline__ void tanh_parts(float v, float* num, float* den) {
  const float u = fabsf(v), z = v * v;
  const float e = __builtin_amdgcn_exp2f(-2.8853900817779268f * u);
  float p = __builtin_fmaf(z, 62.0f / 2835.0f, -17.0f / 315.0f);
  p = __builtin_fmaf(z, p, 2.0f / 15.0f);
  p = __builtin_fmaf(z, p, -1.0f / 3.0f);
  const bool near = u < 0.25f;
  *num = near ? __builtin_fmaf(u * z, p, u) : 1.0f - e;
  *den = near ? 1.0f : 1.0f + e;
}

// SiTU(g, u) = (beta tanh(g / beta) sigmoid(g)) * (lambda tanh(u / lambda)), its three
// quotients over one denominator: three exponentials and one reciprocal, which take four
// issue slots each, are most of a short product's epilogue.  Beta and lambda each go to their
// own quotient's numerator: beta * lambda alone may leave fp32's range where SiTU does not
// (both at 1e20 make it nearly g sigmoid(g) * u).
__device__ __forceinline__ float situ_f32(float g, float u, float beta, float inv_beta, float lam,
                                          float inv_lam) {
  const float a = g * inv_beta, b = u * inv_lam;
  float na, da, nb, db;
  tanh_parts(a, &na, &da);
  tanh_parts(b, &nb, &db);
  const float ds = 1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * g);
  const float mag = (beta * na) * (lam * nb) * __builtin_amdgcn_rcpf(da * db * ds);
  return __uint_as_float(__float_as_uint(mag) ^
                         ((__float_as_uint(a) ^ __float_as_uint(b)) & 0x80000000u));
}

__device__ __forceinline__ float uniform(float v) {
  return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(v)));
}

// A lane's share of a finished tile: its output columns, in groups of four, of M token rows.
// Scales, activation, one rounding to BF16.
template <int Q, bool SITU, int C, int M>
struct Epilogue {
  const GroupedArgs& a;
  int n0[C];                             // first column of each group
  float ws[C][4], us[C][4];              // column scales (us: the up columns with SiTU)
  int row[M];                            // output row, or -1 (not stored)
  float xs[M];                           // row scale
  bool there[M];                         // the row has a source (zeros are stored otherwise)
  float beta, ib, lam, il;               // SiTU

  __device__ __forceinline__ Epilogue(const GroupedArgs& args) : a(args) {}
  // Everything from memory up front: cols(c) is the first column of group c, rows(m) the
  // output row of token m, or -1.
  template <class Cols, class Rows>
  __device__ __forceinline__ void begin(int expert, Cols cols, Rows rows) {
    int64_t src[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
      row[m] = rows(m);
      src[m] = row[m] < 0 ? -1 : source_row(a, row[m]);
    }
#pragma unroll
    for (int m = 0; m < M; ++m) {
      there[m] = src[m] >= 0;
      xs[m] = Q == 0 ? 1.0f : a.x_scale[there[m] ? src[m] : 0];
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      n0[c] = cols(c);
      if constexpr (Q != 0) {
        const float* w = a.w_scale + static_cast<int64_t>(expert) * a.Nw;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = min(n0[c] + i, a.N - 1);
          ws[c][i] = w[n];
          if constexpr (SITU) us[c][i] = w[a.N + n];
        }
      }
    }
    if constexpr (SITU) {
      // the same in every lane: kept in scalar registers
      beta = uniform(a.beta ? a.beta[expert] : 4.0f);
      lam = uniform(a.lam ? a.lam[expert] : 25.0f);
      ib = uniform(1.0f / beta);
      il = uniform(1.0f / lam);
    }
  }
  // Columns of group c of token m: h the (gate) products, u the up products (SiTU).
  __device__ __forceinline__ uint2 columns(int c, int m, typename AccOf<Q>::type h,
                                           typename AccOf<Q>::type u) const {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = static_cast<float>(h[i]);
      if constexpr (Q != 0) v[i] = v[i] * xs[m] * ws[c][i];
      if constexpr (SITU) {
        float uv = static_cast<float>(u[i]);
        if constexpr (Q != 0) uv = uv * xs[m] * us[c][i];
        v[i] = situ_f32(v[i], uv, beta, ib, lam, il);
      }
      if (!there[m]) v[i] = 0.0f;
    }
    return make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  }
  // Store group c, or the adjacent groups c and c + 1.  Where N is no multiple of 4 a row's
  // columns are not aligned to a group and go one by one, which costs the more the shorter K is:
  // 64 experts x 512 rows, K = 512, int8, N = 3584 121 us, N = 3585 317 us; 8 experts x 4096
  // rows, K = 4096, E4M3 414 and 584 us; 896 experts x 18 rows, K = 384, BF16 440 and 491 us.
  __device__ __forceinline__ void store(int c, int m, uint2 v) const {
    uint16_t* o = a.out + static_cast<int64_t>(row[m]) * a.N + n0[c];
    if (a.N % 4 == 0 && n0[c] + 4 <= a.N) {
      *reinterpret_cast<uint2*>(o) = v;
    } else {
      const uint32_t w[2] = {v.x, v.y};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n0[c] + i < a.N) o[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
    }
  }
  __device__ __forceinline__ void store(int c, int m, uint2 lo, uint2 hi) const {
    if (a.N % 8 == 0 && n0[c] + 8 <= a.N) {
      *reinterpret_cast<u32x4*>(a.out + static_cast<int64_t>(row[m]) * a.N + n0[c]) =
          u32x4{lo.x, lo.y, hi.x, hi.y};
    } else {
      store(c, m, lo);
      store(c + 1, m, hi);
    }
  }
};

}  // namespace rmoe
