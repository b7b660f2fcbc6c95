// tiles.hpp -- which workgroup takes which tile, in plain C++: the kernels use it, and
// it compiles for a CPU alone.
#pragma once

#include <cstdint>

#ifdef __HIPCC__
#define TBE_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define TBE_HOST_DEVICE inline
#endif

namespace tbe {

// Tile number q of a group's na x nb tiles: bands of 8 along nb, so that what an XCD
// works on at one time shares operand tiles in its L2.
TBE_HOST_DEVICE void band_order(int64_t q, int64_t na, int64_t nb, int64_t* ta, int64_t* tb) {
  constexpr int64_t kBand = 8;
  const int64_t band = q / (kBand * na), r = q - band * kBand * na;
  const int64_t height = nb - band * kBand < kBand ? nb - band * kBand : kBand;
  *ta = r / height;
  *tb = band * kBand + r % height;
}

// The number, of the `total` tiles of all groups, that workgroup id of `blocks` takes;
// false where it has none.  A launch has a workgroup for every tile of groups that follow
// each other: more tiles are of groups that overlap (bad offsets), and then no workgroup
// takes one, as their numbers may pass every type here.  Workgroups go round robin to the
// 8 XCDs; each XCD takes a contiguous range of the tiles.
TBE_HOST_DEVICE bool tile_number(uint32_t id, uint32_t blocks, int64_t total, int64_t* q) {
  if (static_cast<int64_t>(id) >= total || total > static_cast<int64_t>(blocks)) return false;
  const int64_t xcd = id % 8, rest = total % 8;
  *q = xcd * (total / 8) + (xcd < rest ? xcd : rest) + id / 8;
  return true;
}

}  // namespace tbe
