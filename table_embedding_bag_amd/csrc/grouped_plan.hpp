// grouped_plan.hpp -- which tiles the grouped linear layer's products take, from a call's
// sizes alone.  Plain C++, which compiles for a CPU alone too.
#pragma once

#include <algorithm>
#include <cstdint>

#include "tbe.h"

namespace tbe {

inline int64_t ceil_div(int64_t n, int64_t d) { return (n + d - 1) / d; }

// Rows of operands: of whole 16-byte chunks at aligned addresses; starting at
// multiples of 4 bytes; or, of 2-byte values, at any.
enum RowLayout { kOddRows, kWordRows, kChunkRows };
inline RowLayout row_layout(uintptr_t p, int64_t stride, int64_t width, int64_t bytes) {
  if (p % 16 == 0 && stride * bytes % 16 == 0 && width * bytes % 16 == 0) return kChunkRows;
  return p % 4 == 0 && stride * bytes % 4 == 0 ? kWordRows : kOddRows;
}

// The time of so many equal tiles, in hundredths of a large one's of 2-byte rows.  A CU
// has one tile of 256 at a time or two smaller ones, which take a fifth longer for the
// same outputs, for which they read twice the LDS bytes.  Of fp32 the matrix cores bound all, and the tiles
// of a CU share them; small tiles are a tenth slower for the same outputs.  Large ones
// are no faster (both gradients of 32768 rows in 16 groups, 4096 -> 4096: 16.0 ms, 16.1
// with 128; 8192 in 20, 2048 -> 2048: 1.20, 1.19) and leave more of the last round idle
// (16384 x 1024 -> 1024: 289 us, 257 with 128, 292 with 64): fp32 takes none.
inline int64_t tile_rounds(int tile, int64_t tiles, int32_t dtype) {
  if (dtype == TBE_F32) return (tiles + 255) / 256 * (tile == 128 ? 25 : 7);
  if (tile == 256) return (tiles + 255) / 256 * 100;
  return (tiles + 511) / 512 * (tile == 128 ? 62 : 31);
}

// How the weights' gradient is summed.
struct GradWPlan {
  int tile;           // 256, 128 or 64 outputs on a side
  int64_t chunk;      // groups of more rows are summed in chunks of so many (0: never)
  int64_t slots;      // sums of chunks
};
inline GradWPlan plan_grad_w(int64_t rows, int64_t groups, int64_t K, int64_t M, int32_t dtype) {
  const auto tiles = [&](int64_t t) { return ceil_div(M, t) * ceil_div(K, t); };
  // Large tiles of 2-byte rows are a fifth faster, but need some for each CU: groups
  // differ in size, and the last round leaves CUs idle.  (16384 rows in 8 groups of very
  // different sizes, 1024 x 4096, bf16: 512 large tiles 320 us, 2048 small ones 170.)
  // A single group's are all the same.
  if (dtype != TBE_F32 &&
      (groups * tiles(256) >= 1024 ||
       (groups == 1 && tiles(256) >= 128 &&
        tile_rounds(256, tiles(256), dtype) < tile_rounds(128, tiles(128), dtype))))
    return {256, 0, 0};
  if (groups * tiles(128) >= 512 || rows == 0) return {128, 0, 0};
  // Too few tiles for the chip: chunks of rows, about one for each place.  Where
  // those of 128 outputs would be short, 64: 8191 rows in 5 groups, 250 x 130, fp32,
  // 148 chunk tiles of 128 25 us, 828 of 64 20 us.
  GradWPlan p{rows * tiles(128) < 512 * 256 ? 64 : 128, 0, 0};
  const int64_t places = p.tile == 64 ? 1024 : 512, least = dtype == TBE_F32 ? 128 : 256;
  const int64_t want = ceil_div(rows * tiles(p.tile), places);
  p.chunk = std::max(least, (want + 63) / 64 * 64);
  // a group of n > chunk rows has at most 2 n / chunk chunks
  p.slots = rows > p.chunk ? 2 * rows / p.chunk : 0;
  return p;
}

// The tiles of a product over rows, by their outputs along the columns.  32 stands
// for those of 128 x 32, for groups of few rows, whose weights' reading is what counts
// (64 rows over 64 groups, 512 -> 2048 bf16: 18 us, 21 with the others; 4096 rows: 35
// with 128, 41 with 64).  Of the others the one with the fewest rounds of tiles by the
// time of a round (tile_rounds), which agrees with these, in us (2-byte rows):
//   16384 rows in 8 groups, 1024 -> 4096   256 162, 128 177
//   16384 rows in 8 groups, 4096 -> 1024   256 183, 128 172
//   8192 rows in 8 groups, 1024 -> 1024    256 30, 128 32, 64 41
//   4096 rows in 8 groups, 1024 -> 1024    256 26, 128 22, 64 25
//   2048 rows in 8 groups, 1024 -> 512     128 14, 64 11
// and of fp32, 1266 rows in 2 groups, 384 -> 4032, 128 61, 64 55.
inline int64_t row_rounds(int64_t rows, int64_t groups, int64_t cols, int tile, int32_t dtype) {
  // a group's last tile is half full on the average
  const int64_t tiles = groups == 1 ? ceil_div(rows, tile) : rows / tile + groups / 2;
  return tile_rounds(tile, tiles * ceil_div(cols, tile), dtype);
}
inline int row_tile(int64_t rows, int64_t groups, int64_t cols, int32_t dtype) {
  if (rows <= groups * 32) return 32;
  const auto rounds = [&](int tile) { return row_rounds(rows, groups, cols, tile, dtype); };
  const int small = rounds(64) <= rounds(128) ? 64 : 128;
  return dtype != TBE_F32 && rounds(256) < rounds(small) ? 256 : small;
}

// The tiles of both gradients, and whether they share a launch, where dx is wanted.
struct BackwardPlan {
  GradWPlan w;
  bool both;
};
inline BackwardPlan plan_backward(int64_t rows, int64_t groups, int64_t K, int64_t M, bool dx,
                                  int32_t dtype) {
  BackwardPlan p{plan_grad_w(rows, groups, K, M, dtype), false};
  // The one launch makes up for rows' tiles that take longer, where the weights' are
  // few and the largest group's last ones run alone: up to half (8192 rows in 8 groups,
  // 1024 -> 1024, 512 tiles, bf16: 55 us, 64 in two launches; fp32 4096 rows 165, 221),
  // else a tenth (8192 rows, 1024 -> 4096 fp32, 2048 tiles: 1273 us, 1162 in two).
  const int best = row_tile(rows, groups, K, dtype);
  if (!dx || best == 32) return p;
  const int64_t own = row_rounds(rows, groups, K, p.w.tile, dtype);
  const int64_t least = row_rounds(rows, groups, K, best, dtype);
  const int64_t tiles = groups * ceil_div(M, p.w.tile) * ceil_div(K, p.w.tile);
  p.both = own * 20 <= least * (tiles < 1024 ? 30 : 22);
  return p;
}

}  // namespace tbe
