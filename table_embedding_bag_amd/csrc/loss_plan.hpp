// loss_plan.hpp -- which tiles, pieces and splits the softmax loss takes, from a call's
// sizes alone.  Plain C++, which compiles for a CPU alone too.
#pragma once

#include <algorithm>
#include <cstdint>

#include "grouped_plan.hpp"

namespace tbe {

// Rows of the workspaces' matrices are whole 128-byte lines.
inline int64_t padded_width(int64_t width, int64_t bytes) {
  const int64_t line = 128 / bytes;
  return ceil_div(width, line) * line;
}

// Whether a table's rows are narrow enough for kernels that keep rows in registers
// (loss_narrow.hpp); such a table may still have to be read by words.
constexpr int64_t kNarrow = 128;
inline bool narrow_rows(int64_t K, int32_t dtype) { return dtype != TBE_F32 && K <= kNarrow && K % 8 == 0; }

// The forward pass: a workgroup has `tile` rows (32: tiles of 128 x 32) and `run`
// consecutive tiles of the vocabulary; a row gets one partial sum of each segment.
// narrow: of a workgroup's waves that have rows of their own, 4 or 1 (0: other kernels).
struct LossForwardPlan {
  int tile, narrow;
  int64_t tiles, run, segments;
};
inline LossForwardPlan plan_loss_forward(int64_t rows, int64_t vocab, int64_t K, bool narrow,
                                         int32_t dtype) {
  LossForwardPlan p{};
  if (narrow) {
    p.narrow = rows <= 64 ? 1 : 4;
    p.tiles = ceil_div(vocab, p.narrow == 1 ? 128 : 64);
    // two workgroups a CU, or one where they share their rows and have larger rings
    const int64_t want = std::max<int64_t>(1, p.narrow == 1 ? 256 : 512 / ceil_div(rows, 256));
    p.run = ceil_div(p.tiles, std::min(want, p.tiles));
    p.segments = ceil_div(p.tiles, p.run);
    return p;
  }
  // (16384 rows, 131072 outputs of 512, fp16: 2.20 ms with 256, 2.70 with 128; 3000 rows, 20001
  // of 513: 103 us, 138.)
  p.tile = rows <= 32 ? 32 : row_tile(vocab, 1, rows, dtype);
  const int64_t along_rows = ceil_div(rows, p.tile);
  p.tiles = ceil_div(vocab, p.tile == 32 ? 128 : p.tile);
  // workgroups for every place of the chip, twice over
  const int64_t want = std::max<int64_t>(1, (p.tile == 256 ? 512 : 1024) / along_rows);
  p.run = ceil_div(p.tiles, std::min(want, p.tiles));
  p.segments = ceil_div(p.tiles, p.run);
  return p;
}

// One gradient's product of a piece: outputs [out_rows, K], summed over `depth`.
struct LossProductPlan {
  int tile;
  int64_t splits, each;  // parts of the summed index, values in each
};
inline LossProductPlan plan_loss_product(int64_t out_rows, int64_t K, int64_t depth, int32_t dtype) {
  const auto tiles = [&](int64_t t) { return ceil_div(out_rows, t) * ceil_div(K, t); };
  LossProductPlan p{};
  // Few outputs over a short index take small tiles (the backward pass of 700 rows, 3000
  // outputs of 1000, fp16: 53 us, 67 with 128; of 4096 rows, 20000 of 256: 249, 225 with 128).
  p.tile = dtype != TBE_F32 && K > 128 && tiles(256) >= 128 ? 256
           : depth * tiles(128) < 512 * 384                 ? 64
                                                            : 128;
  const int64_t places = p.tile == 256 ? 256 : p.tile == 128 ? 512 : 1024;
  const int64_t want = std::max<int64_t>(1, places / tiles(p.tile));
  p.each = std::max<int64_t>(128, ceil_div(ceil_div(depth, want), 64) * 64);
  p.splits = ceil_div(depth, p.each);
  return p;
}

// A gradient's kernel of narrow rows: workgroups of 256 output rows, the other side's
// tiles of 64 rows in parts of `run`.
struct LossNarrowPlan {
  int64_t splits, run;
};
inline LossNarrowPlan plan_loss_narrow(int64_t out_rows, int64_t other_rows) {
  const int64_t tiles = ceil_div(other_rows, 64);
  const int64_t want = std::max<int64_t>(1, 256 / ceil_div(out_rows, 256));
  LossNarrowPlan p{};
  p.run = ceil_div(tiles, std::min(want, tiles));
  p.splits = ceil_div(tiles, p.run);
  return p;
}

// The backward pass goes over the vocabulary in pieces of `piece` rows of the table.
struct LossBackwardPlan {
  int tile;               // of the logits
  int64_t piece, pieces;
  int64_t width;          // of a row of the piece's gradients of the logits
  LossProductPlan x, w;   // of a whole piece
  bool narrow;
  LossNarrowPlan nx, nw;  // where narrow, instead of all that
};
inline LossBackwardPlan plan_loss_backward(int64_t rows, int64_t vocab, int64_t K, bool narrow,
                                           int32_t dtype) {
  LossBackwardPlan p{};
  p.narrow = narrow;
  if (narrow) {
    p.nx = plan_loss_narrow(rows, vocab);
    p.nw = plan_loss_narrow(vocab, rows);
    return p;
  }
  const int64_t bytes = dtype == TBE_F32 ? 4 : 2;
  const int64_t most = std::max<int64_t>(int64_t{1} << 10, (int64_t{512} << 20) / (rows * bytes));
  const int64_t n = ceil_div(vocab, std::min<int64_t>(most, int64_t{1} << 18));
  p.piece = std::min(vocab, ceil_div(ceil_div(vocab, n), 256) * 256);
  p.pieces = ceil_div(vocab, p.piece);
  p.width = padded_width(p.piece, bytes);
  p.tile = std::max(64, row_tile(p.piece, 1, rows, dtype));
  p.x = plan_loss_product(rows, K, p.piece, dtype);
  p.w = plan_loss_product(p.piece, K, rows, dtype);
  return p;
}

}  // namespace tbe
