// Device helpers of the products grouped by expert of microscaled FP4 rows (grouped_mxfp4.hip,
// grouped_mxfp4_big.hip).
#pragma once

#include "common.h"
#include "grouped.h"
#include "grouped_mxfp4_rule.h"
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

// Where loads into LDS read an operand.  Loads through a buffer descriptor take a 32-bit offset
// per lane and one for all lanes, and give zeros for an offset past its end (kNowhere): a load is
// one instruction behind the one that says where in LDS, its lanes' ends of K one more.  With
// addresses of 64 bits (WIDE, for operands of 4 GB and more: a workgroup's weights are one
// expert's, and its token rows those of a tile where nothing gathers them) it is three or four more,
// and a chunk's loads were most of what a wavefront did.
typedef __amdgpu_buffer_rsrc_t buffer_t;
constexpr uint32_t kNowhere = kMxBufferMost;
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

}  // namespace rmoe
