// The grouped linear layer's tile arithmetic (csrc/tiles.hpp, csrc/grouped_plan.hpp) on the CPU:
// which tiles a call takes, and the tile of the groups' rows that each workgroup of a launch finds.
#include <algorithm>
#include <cstdint>
#include <vector>

#include "grouped_plan.hpp"
#include "tiles.hpp"

extern "C" {

// Workgroups 0 .. blocks - 1 of a product over rows: TB rows a tile, na tiles along the other
// index.  Returns the workgroups that have a tile, or -1 where one starts outside its group's
// rows; lowest and highest: of the rows that tiles hold.  taken [tiles of all groups]: how often
// each was taken (null: not wanted).
int64_t row_tiles(const int64_t* offsets, int64_t groups, int64_t rows, int64_t blocks, int64_t na,
                  int64_t TB, int64_t* lowest, int64_t* highest, int32_t* taken) {
  std::vector<int64_t> first(groups), n(groups), before(groups + 1);
  for (int64_t g = 0; g < groups; ++g) {
    const auto at = [&](int64_t i) { return std::min(std::max<int64_t>(offsets[i], 0), rows); };
    first[g] = at(g);
    n[g] = std::max<int64_t>(at(g + 1) - at(g), 0);
    before[g + 1] = before[g] + (n[g] + TB - 1) / TB * na;
  }
  const int64_t total = before[groups];
  int64_t count = 0;
  *lowest = rows, *highest = -1;
  for (int64_t id = 0; id < blocks; ++id) {
    int64_t q;
    if (!tbe::tile_number(static_cast<uint32_t>(id), static_cast<uint32_t>(blocks), total, &q)) continue;
    // the kernels take the first group whose tiles end behind q
    const int64_t g = std::upper_bound(before.begin() + 1, before.end(), q) - before.begin() - 1;
    if (g >= groups) continue;
    int64_t ta, tb;
    tbe::band_order(q - before[g], na, (n[g] + TB - 1) / TB, &ta, &tb);
    ++count;
    if (ta < 0 || ta >= na || tb < 0 || tb * TB >= n[g]) return -1;
    *lowest = std::min(*lowest, first[g] + tb * TB);
    *highest = std::max(*highest, first[g] + std::min(n[g], (tb + 1) * TB) - 1);
    if (taken) ++taken[before[g] + tb * na + ta];
  }
  return count;
}

// The tiles of a call's products: {forward, dx, dweight, its chunk, its slots, whether dx and
// dweight share a launch}.
void plan(int64_t rows, int64_t groups, int64_t K, int64_t M, int32_t dx, int32_t dtype, int64_t* out) {
  const tbe::BackwardPlan b = tbe::plan_backward(rows, groups, K, M, dx != 0, dtype);
  out[0] = tbe::row_tile(rows, groups, M, dtype);
  out[1] = tbe::row_tile(rows, groups, K, dtype);
  out[2] = b.w.tile;
  out[3] = b.w.chunk;
  out[4] = b.w.slots;
  out[5] = b.both;
}

// The layout of an operand's rows (0 odd, 1 words, 2 chunks).
int32_t layout(uint64_t address, int64_t stride, int64_t width, int64_t bytes) {
  return tbe::row_layout(static_cast<uintptr_t>(address), stride, width, bytes);
}

// The time of a product's tiles in hundredths of a large tile's.
int64_t rounds(int64_t rows, int64_t groups, int64_t cols, int32_t tile, int32_t dtype) {
  return tbe::row_rounds(rows, groups, cols, tile, dtype);
}

}  // extern "C"
