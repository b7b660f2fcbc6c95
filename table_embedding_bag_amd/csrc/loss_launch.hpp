// loss_launch.hpp -- which of the softmax loss's kernels a call takes.
#pragma once

#include "loss_kernels.hpp"
#include "loss_narrow.hpp"

namespace tbe {
namespace {

using LossLarge = Shape<256, 256, 2, 4, 2, 128>;
using LossMedium = Shape<128, 128, 2, 2, 2, 128>;
// Rows are a few slices long, so that more workgroups a CU count for more than slices in flight
// (us with 4, 3, 2 slices: 1000 rows, 9973 outputs of 100, fp32, both directions 149, 138, 134;
// backward, 700 rows, 3000 of 1000, fp16 57, 53, 55; 300 rows, 5000 of 200, fp16 50, 41, 47).
template <int ST>
using LossSquare = Shape<64, 64, 2, 2, ST == kF32 ? 2 : 3, 128>;
using LossSlim = Shape<128, 32, 4, 1, 4, 128>;

// f(the layout, known to the compiler)
template <int ST, typename F>
void with_rows(int32_t layout, F f) {
  if (layout == kChunkRows) return f(std::integral_constant<int, kChunkRows>{});
  if constexpr (StorageTraits<ST>::bytes == 2)
    if (layout == kOddRows) return f(std::integral_constant<int, kOddRows>{});
  f(std::integral_constant<int, kWordRows>{});
}

// f(the shape of tiles of so many rows)
template <int ST, typename F>
void with_tile(int tile, F f) {
  if constexpr (ST != kF32)
    if (tile == 256) return f(LossLarge{});
  if (tile == 64) return f(LossSquare<ST>{});
  f(LossMedium{});
}

// f(slices of 64 values in a narrow row, known to the compiler)
template <typename F>
void with_slices(int64_t K, F f) {
  if (K <= 64) f(std::integral_constant<int, 1>{});
  else f(std::integral_constant<int, 2>{});
}

// A gradient's parts to the gradient.
template <int ST>
hipError_t launch_loss_sum(const LossArgs& a, const float* parts, int64_t splits, int64_t n, void* out,
                           hipStream_t s) {
  hipLaunchKernelGGL((loss_sum<ST>), dim3(static_cast<unsigned>(ceil_div(ceil_div(n, 4), kBlock))),
                     dim3(kBlock), 0, s, a, parts, splits, n, out);
  return hipGetLastError();
}

template <int ST, bool DTABLE>
hipError_t launch_loss_narrow(const LossArgs& a, hipStream_t s) {
  const LossNarrowPlan& p = DTABLE ? a.backward.nw : a.backward.nx;
  const int64_t out_rows = DTABLE ? a.vocab : a.rows;
  void* out = DTABLE ? a.dtable : a.dx;
  float* parts = DTABLE ? a.dw_parts : a.dx_parts;
  with_slices(a.K, [&](auto slices) {
    using S = NarrowShape<slices, 4, 2>;
    hipLaunchKernelGGL((loss_narrow_gradient<ST, S, DTABLE>),
                       dim3(static_cast<unsigned>(ceil_div(out_rows, S::QR) * p.splits)), dim3(kBlock), 0, s,
                       a, p.splits, p.run, parts, parts ? nullptr : out);
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !parts) return e;
  return launch_loss_sum<ST>(a, parts, p.splits, out_rows * a.K, out, s);
}

template <int ST>
hipError_t launch_loss_forward(const LossArgs& a, hipStream_t s) {
  if constexpr (ST != kF32) {
    if (a.forward.narrow)
      with_slices(a.K, [&](auto slices) {
        const auto go_narrow = [&](auto shape) {
          using S = decltype(shape);
          hipLaunchKernelGGL((loss_narrow_forward<ST, S>),
                             dim3(static_cast<unsigned>(ceil_div(a.rows, S::QR) * a.forward.segments)),
                             dim3(kBlock), 0, s, a);
        };
        if (a.forward.narrow == 1) go_narrow(NarrowShape<slices, 1, 1>{});
        else go_narrow(NarrowShape<slices, 4, 2>{});
      });
  }
  const auto go = [&](auto shape) {
    using S = decltype(shape);
    const int64_t blocks = ceil_div(a.rows, S::TB) * a.forward.segments;
    with_rows<ST>(a.layout, [&](auto layout) {
      hipLaunchKernelGGL((loss_forward<ST, S, layout>), dim3(static_cast<unsigned>(blocks)),
                         dim3(S::threads), 0, s, a);
    });
  };
  if (a.forward.narrow) {}
  else if (a.forward.tile == 32) go(LossSlim{});
  else with_tile<ST>(a.forward.tile, go);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((loss_join<ST>), dim3(static_cast<unsigned>(ceil_div(a.rows, 16))), dim3(kBlock), 0,
                     s, a);
  return hipGetLastError();
}

template <int ST, bool TABLE>
hipError_t launch_loss_product(const LossArgs& a, int64_t v0, int64_t piece, const LossProductPlan& plan,
                               int32_t add, hipStream_t s) {
  const int64_t out_rows = TABLE ? piece : a.rows, depth = TABLE ? a.rows : piece;
  const int64_t splits = ceil_div(depth, plan.each);
  void* out = TABLE && plan.splits == 1 ? a.dtable : nullptr;
  with_tile<ST>(plan.tile, [&](auto shape) {
    using S = decltype(shape);
    const int64_t blocks = ceil_div(a.K, S::TA) * ceil_div(out_rows, S::TB) * splits;
    const auto go = [&](auto layout) {
      hipLaunchKernelGGL((loss_product<ST, S, layout, TABLE>), dim3(static_cast<unsigned>(blocks)),
                         dim3(S::threads), 0, s, a, v0, piece, splits, plan.each, out, add);
    };
    if constexpr (TABLE) go(std::integral_constant<int, kChunkRows>{});
    else with_rows<ST>(a.table_layout, go);
  });
  hipError_t e = hipGetLastError();
  if (!TABLE || out || e != hipSuccess) return e;
  return launch_loss_sum<ST>(a, a.dw_parts, splits, piece * a.K,
                             static_cast<char*>(a.dtable) + v0 * a.K * StorageTraits<ST>::bytes, s);
}

template <int ST>
hipError_t launch_loss_backward(const LossArgs& a, hipStream_t s) {
  constexpr int E = 16 / StorageTraits<ST>::bytes;
  if constexpr (ST == kF16) {
    hipLaunchKernelGGL(loss_factor, dim3(1), dim3(1024), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int64_t chunks = std::max<int64_t>(1, a.rows * (a.x_width / E));
  hipLaunchKernelGGL((loss_prepare<ST>),
                     dim3(static_cast<unsigned>(std::min<int64_t>(ceil_div(chunks, kBlock), 4096))),
                     dim3(kBlock), 0, s, a);
  hipError_t e = hipGetLastError();
  if (a.rows == 0) {  // no rows: a gradient of zeros
    const int64_t all = a.vocab * a.K, most = int64_t{1} << 30;
    for (int64_t v = 0; e == hipSuccess && v < all; v += most) {
      const int64_t n = std::min(most, all - v);
      e = launch_loss_sum<ST>(a, nullptr, 0, n, static_cast<char*>(a.dtable) + v * StorageTraits<ST>::bytes, s);
    }
    return e;
  }
  if constexpr (ST != kF32) {
    if (a.backward.narrow) {
      if (e == hipSuccess && a.dtable) e = launch_loss_narrow<ST, true>(a, s);
      if (e == hipSuccess && a.dx) e = launch_loss_narrow<ST, false>(a, s);
      return e;
    }
  }
  for (int64_t v0 = 0; e == hipSuccess && v0 < a.vocab; v0 += a.backward.piece) {
    const int64_t piece = std::min(a.backward.piece, a.vocab - v0);
    with_tile<ST>(a.backward.tile, [&](auto shape) {
      using S = decltype(shape);
      const int64_t blocks = ceil_div(a.rows, S::TB) * ceil_div(piece, S::TA);
      with_rows<ST>(a.layout, [&](auto layout) {
        hipLaunchKernelGGL((loss_dlogits<ST, S, layout>), dim3(static_cast<unsigned>(blocks)),
                           dim3(S::threads), 0, s, a, v0, piece);
      });
    });
    e = hipGetLastError();
    if (e == hipSuccess && a.dtable) e = launch_loss_product<ST, true>(a, v0, piece, a.backward.w, 0, s);
    if (e == hipSuccess && a.dx) e = launch_loss_product<ST, false>(a, v0, piece, a.backward.x, v0 > 0, s);
  }
  if (e != hipSuccess || !a.dx) return e;
  return launch_loss_sum<ST>(a, a.dx_parts, a.backward.x.splits, a.rows * a.K, a.dx, s);
}

template <int ST>
hipError_t launch_loss(const LossArgs& a, bool backward, hipStream_t s) {
  return backward ? launch_loss_backward<ST>(a, s) : launch_loss_forward<ST>(a, s);
}

}  // namespace
}  // namespace tbe
