// Which kernel a call of the products by expert of microscaled FP4 rows takes.  Plain host code: the
// launch (grouped_mxfp4.hip) uses it, and a test asks it which kernels its problems reach.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

namespace rmoe {

// The largest operand that a buffer descriptor's 32-bit offsets reach (kNowhere lies behind it).
constexpr uint32_t kMxBufferMost = 0xFFFF0000u;
// A list of source rows in LDS holds at most so many.
constexpr int kMxListRows = 2048;
constexpr size_t kMxLdsBytes = 163840;

struct MxSizes {
  int64_t R, E, Nw, KB, x_rows;  // KB: code bytes of a row
  bool gathered;                 // rows through row_idx
  int cus;
};

// Tiles of 256 x 256, or of up to `rows` rows by 32 `waves` weight rows, `per_cu` workgroups on a CU;
// wide: with 64-bit addresses.
struct MxTiles {
  int rows, waves, per_cu;
  bool wide;
};
constexpr MxTiles kMxBig{256, 4, 1, false};
constexpr int kMxRing = 3;       // chunks in LDS of the smaller ones

// Operands past what a buffer descriptor reaches.
inline bool mx_wide(const MxSizes& s) {
  return static_cast<uint64_t>(s.Nw) * s.KB > kMxBufferMost ||
         (s.gathered && static_cast<uint64_t>(s.x_rows) * s.KB > kMxBufferMost);
}

// Larger tiles read the weights for more rows at once; smaller ones and smaller blocks of weight rows
// make more work items.  items() is an upper bound of the items of a kernel (the host does not know
// the rows of each expert), `few` three quarters of the CUs.  Measured on one MI355X, us with tiles
// of 256 / 128 / 64 rows by 256 weight rows, 64 by 128, 32 by 64 and 16 by 64:
//   many rows per expert: 64 experts x 512 rows, N = K = 2048  130 / 146 / 190 / 183 / 287 / 438;
//     x 256 rows (half of the experts above one tile)  80 / 84 / 103 / 100 / 157 / 230, but 896 x
//     292 rows, N = 384 with SiTU, K = 3584  986 / 872 / 1138 / 1373 / 2282 / 2614; 8 x 256 rows,
//     N = K = 4096, whose tiles of 256 are one round of the chip  43 / 55 / 58 / 52 / 76 / 109;
//   fewer: 896 x 73 rows, the same N and K  440 / 347 / 458 / 522 / 707 / 798; 18 rows, N = 3584,
//     K = 384, Zipf  345 / 216 / 210 / 284 / 321 / 251; 4.6 rows  288 / 202 / 186 / 240 / 237 / 158;
//     1.1 rows, N = 384 with SiTU, K = 3584  112 / 77 / 76 / 85 / 83 / 72;
//   few items: 8 experts x 32 rows, N = K = 4096  26 / 24 / 24 / 18 / 24 / 28; one expert, N = K =
//     7168, 512 rows  52 / 46 / 36 / 36 / 52 / 81, 64 rows  34 / 34 / 33 / 21 / 15 / 17, 16 rows
//     33 / 29 / 28 / 18 / 13 / 13;
//   rows that all fall on one of 896 experts, which the host does not know and the rule takes for few
//     rows each: N = 384 with SiTU, K = 3584, 16384 rows 60 us (called with one expert 53), 4096 rows
//     37 (23).
inline MxTiles mx_tiles(const MxSizes& s) {
  const int64_t R = s.R, E = s.E, some = std::min(R, E), few = s.cus * 3 / 4;
  auto items = [&](int tile, int block) { return (some + R / tile) * ((s.Nw + block - 1) / block); };
  // (operands past the descriptors' reach, whose loads cost more, are not worth more kernels than two)
  if (mx_wide(s)) return R > 8 * some ? MxTiles{64, 4, 2, true} : MxTiles{16, 2, 4, true};
  // (the LDS of the larger tiles leaves room for so many experts' prefix sums)
  const int64_t items256 = items(256, 256);
  if (E <= 1024 && items256 >= few && (R >= 448 * E || (R >= 224 * E && items256 <= s.cus)))
    return kMxBig;
  if (items(128, 256) >= few) {
    if (E <= 1536 && R > 32 * E) return MxTiles{128, 8, 1, false};
    if (E <= 8192 && R > 8 * E) return MxTiles{64, 8, 1, false};
    if (R > 8 * E) return MxTiles{64, 4, 2, false};
  } else if (R > 16 * some) {
    if (items(64, 128) >= few) return MxTiles{64, 4, 2, false};
    return MxTiles{32, 2, 4, false};
  }
  return MxTiles{16, 2, 4, false};
}

// LDS bytes of a ring of the smaller tiles: codes and scales of the weight rows and token rows (the
// latter's scales at least 32 rows at a time).
constexpr size_t mx_ring_bytes(const MxTiles& t) {
  return kMxRing * ((32 * t.waves + t.rows) * size_t(128) + (32 * t.waves + std::max(t.rows, 32)) * size_t(8));
}

// Whether the smaller tiles read their source rows from row_idx itself: where there are too many for a
// list in LDS, or it does not fit behind the ring and the prefix sums (less what the scan takes).
inline bool mx_direct(const MxSizes& s, const MxTiles& t) {
  return s.gathered && (s.R > kMxListRows ||
                        mx_ring_bytes(t) + (s.E + 1) * 4 + s.R * 4 > kMxLdsBytes - 128);
}

}  // namespace rmoe
