// softmax_loss.hpp -- kernels of the softmax loss (softmax_loss.hip has the interface;
// softmax_loss_f32/f16/bf16.hip each compile them for one type).
#pragma once

#include "layers.hpp"
#include "loss_plan.hpp"
#include "tiles.hpp"
#ifdef TBE_LOSS_KERNELS
#include "products.hpp"
#endif

namespace tbe {

struct LossArgs {
  int64_t rows, vocab, K;
  const void* x;
  const void* table;
  const void* targets;
  int64_t x_stride, table_stride;
  int32_t index64;
  int32_t layout;         // of x and the table together
  int32_t table_layout;   // of the table
  float scale;            // logits = scale x W^T
  float exponent;         // scale log2(e): of the powers of two
  // forward
  LossForwardPlan forward;
  float2* parts;          // [segments][rows]: a row's largest exponent and its sum of powers
  float* target_logit;    // [rows], before the scale; rows without a target: not written
  float* loss;
  float* lse;
  // backward
  LossBackwardPlan backward;
  const float* lse_in;
  const float* grad;      // [rows]
  void* x_rows;           // [rows][x_width]: x, zeros where a row has no target; or null
  int64_t x_width;
  void* dlogits;          // [rows][backward.width]: of one piece
  float* dx_parts;        // [backward.x.splits][rows][K]
  float* dw_parts;        // [backward.w.splits][piece][K], or null with one split
  float* factor;          // {what the logits' gradients are multiplied by, what undoes it times scale}
  void* dx;               // or null
  void* dtable;           // or null
};

hipError_t launch_loss_f32(const LossArgs& a, bool backward, hipStream_t s);
hipError_t launch_loss_f16(const LossArgs& a, bool backward, hipStream_t s);
hipError_t launch_loss_bf16(const LossArgs& a, bool backward, hipStream_t s);

#ifdef TBE_LOSS_KERNELS

namespace {

constexpr float kNegInf = -__builtin_inff();

// The target of row n, or -1 where it has none (or one outside the table).
__device__ __forceinline__ int64_t target_of(const LossArgs& a, int64_t n) {
  const int64_t t = a.index64 ? static_cast<const int64_t*>(a.targets)[n]
                              : static_cast<const int32_t*>(a.targets)[n];
  return t >= 0 && t < a.vocab ? t : -1;
}

// Which of a wave's 16 WA logits of a row the lane's i-th fragment's e-th value is.
__device__ __forceinline__ int place_of(int i, int e, int lane) {
  return 32 * i + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
}

// The logits of a tile (before the scale): acc[i][j][e] of row 32 j + lane % 32 and
// vocabulary row place_of(i, e, lane) of the wave's outputs.
template <int ST, typename S, int LAYOUT>
__device__ __forceinline__ void tile_logits(const LossArgs& a, int64_t v0, int64_t vocab_left,
                                            const void* x, int64_t x_stride, int64_t n0, int wa,
                                            int wb, int wave, int lane, unsigned char* lds,
                                            f32x16 (&acc)[S::WA][S::WB]) {
  constexpr int bytes = StorageTraits<ST>::bytes, kAhead = kHeldSlices<S, LAYOUT>;
  Operand<ST, true, S::TA, S::NW, LAYOUT, S::RB, kAhead> oa;
  Operand<ST, true, S::TB, S::NW, LAYOUT, S::RB, kAhead> ob;
  oa.init(static_cast<const char*>(a.table) + v0 * a.table_stride * bytes, a.table_stride, vocab_left,
          a.K, wave, lane);
  ob.init(static_cast<const char*>(x) + n0 * x_stride * bytes, x_stride, a.rows - n0, a.K, wave, lane);
#pragma unroll
  for (int i = 0; i < S::WA; ++i)
#pragma unroll
    for (int j = 0; j < S::WB; ++j) acc[i][j] = f32x16{};
  accumulate<ST, S, LAYOUT>(oa, ob, a.K, lds, wa, wb, wave, lane, acc, [](const u32x4 (&)[S::WB]) {});
}

// Forward: the running largest exponent m and sum s of 2^(exponent - m) of each row over
// the segment's tiles, lane by lane; joined over lanes and waves once at the end.
template <int ST, typename S, int LAYOUT>
__global__ __launch_bounds__(S::threads) void loss_forward(LossArgs a) {
  __shared__ __align__(1024) unsigned char lds[kLdsBytes<S, LAYOUT>];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wa = (wave % S::NA) * S::WA * 32, wb = (wave / S::NA) * S::WB * 32;
  const int64_t nb = (a.rows + S::TB - 1) / S::TB;
  int64_t segment, tb;
  band_order(xcd_contiguous_block(blockIdx.x, gridDim.x), a.forward.segments, nb, &segment, &tb);
  const int64_t b0 = tb * S::TB;
  const int64_t first = segment * a.forward.run;
  const int64_t last = first + a.forward.run < a.forward.tiles ? first + a.forward.run : a.forward.tiles;
  float m[S::WB], sum[S::WB];
  int64_t target[S::WB];
#pragma unroll
  for (int j = 0; j < S::WB; ++j) {
    m[j] = kNegInf;
    sum[j] = 0.0f;
    const int64_t n = b0 + wb + 32 * j + (lane & 31);
    target[j] = n < a.rows ? target_of(a, n) : -1;
  }
  for (int64_t t = first; t < last; ++t) {
    const int64_t a0 = t * S::TA, left = a.vocab - a0;
    f32x16 acc[S::WA][S::WB];
    if (t > first) __syncthreads();  // the tile before is read
    tile_logits<ST, S, LAYOUT>(a, a0, left, a.x, a.x_stride, b0, wa, wb, wave, lane, lds, acc);
    if (left < S::TA) {  // the last: nothing past the table's end
#pragma unroll
      for (int i = 0; i < S::WA; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (wa + place_of(i, e, lane) >= left)
#pragma unroll
            for (int j = 0; j < S::WB; ++j) acc[i][j][e] = kNegInf;
    }
#pragma unroll
    for (int j = 0; j < S::WB; ++j) {
      const int64_t at = target[j] - a0 - wa;
      if (__any(target[j] >= 0 && at >= 0 && at < 32 * S::WA)) {
#pragma unroll
        for (int i = 0; i < S::WA; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (target[j] >= 0 && at == place_of(i, e, lane))
              a.target_logit[b0 + wb + 32 * j + (lane & 31)] = acc[i][j][e];
      }
      float top = kNegInf;
#pragma unroll
      for (int i = 0; i < S::WA; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) top = fmaxf(top, acc[i][j][e]);
      const float next = fmaxf(m[j], top * a.exponent);
      const float from = next == kNegInf ? 0.0f : next;
      float part[4] = {};
#pragma unroll
      for (int i = 0; i < S::WA; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          part[e & 3] += __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][e], a.exponent, -from));
      sum[j] = sum[j] * __builtin_amdgcn_exp2f(m[j] - from) + ((part[0] + part[1]) + (part[2] + part[3]));
      m[j] = next;
    }
  }
  // the two halves of a wave, then the waves that have the same rows
  __syncthreads();
  float2* joined = reinterpret_cast<float2*>(lds);
#pragma unroll
  for (int j = 0; j < S::WB; ++j) {
    const float m2 = __shfl_xor(m[j], 32), s2 = __shfl_xor(sum[j], 32);
    const float top = fmaxf(m[j], m2), from = top == kNegInf ? 0.0f : top;
    const float s = sum[j] * __builtin_amdgcn_exp2f(m[j] - from) + s2 * __builtin_amdgcn_exp2f(m2 - from);
    if (lane < 32) joined[(wave % S::NA) * S::TB + wb + 32 * j + lane] = make_float2(top, s);
  }
  __syncthreads();
  for (int r = threadIdx.x; r < S::TB; r += S::threads) {
    if (b0 + r >= a.rows) break;
    float2 v = joined[r];
#pragma unroll
    for (int w = 1; w < S::NA; ++w) {
      const float2 o = joined[w * S::TB + r];
      const float top = fmaxf(v.x, o.x), from = top == kNegInf ? 0.0f : top;
      v.y = v.y * __builtin_amdgcn_exp2f(v.x - from) + o.y * __builtin_amdgcn_exp2f(o.x - from);
      v.x = top;
    }
    a.parts[segment * a.rows + b0 + r] = v;
  }
}

// A row's segments joined, 16 rows a workgroup, 16 segments at a time.
template <int ST>
__global__ __launch_bounds__(kBlock) void loss_join(LossArgs a) {
  __shared__ float2 part[16][16];
  const int r = threadIdx.x & 15, slice = threadIdx.x >> 4;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 16 + r;
  float m = kNegInf, s = 0.0f;
  const auto add = [&](float2 o) {
    const float top = fmaxf(m, o.x), from = top == kNegInf ? 0.0f : top;
    s = s * __builtin_amdgcn_exp2f(m - from) + o.y * __builtin_amdgcn_exp2f(o.x - from);
    m = top;
  };
  if (n < a.rows)
#pragma unroll 4
    for (int64_t g = slice; g < a.forward.segments; g += 16) add(a.parts[g * a.rows + n]);
  part[slice][r] = make_float2(m, s);
  __syncthreads();
  if (slice == 0 && n < a.rows) {
    for (int i = 1; i < 16; ++i) add(part[i][r]);
    // in 64 bits: the difference of two large values is what is asked for
    const double ln2 = 0.69314718055994530942;
    const double power = ln2 * (static_cast<double>(m) + static_cast<double>(log2f(s)));
    a.lse[n] = static_cast<float>(power);
    a.loss[n] = target_of(a, n) < 0 ? 0.0f
                                    : static_cast<float>(power - ln2 * static_cast<double>(a.exponent) *
                                                                     static_cast<double>(a.target_logit[n]));
  }
}

// x for the table's gradient: rows without a target are zeros, whatever they hold, and
// so is what follows a row's end.  The first workgroup sets the factors: fp16 gradients
// of the logits are multiplied by 2^14 over the largest row gradient's power of two, so
// that probabilities down to 2^-28 of it stay normal numbers.
template <int ST>
__global__ __launch_bounds__(kBlock) void loss_prepare(LossArgs a) {
  constexpr int E = 16 / StorageTraits<ST>::bytes;
  if (blockIdx.x == 0) {
    __shared__ float part[kWavesPerBlock];
    float top = 0.0f;
    if constexpr (ST == kF16) {
      for (int64_t n = threadIdx.x; n < a.rows; n += kBlock)
        if (target_of(a, n) >= 0) top = fmaxf(top, fabsf(a.grad[n]));
      for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
      if (lane_id() == 0) part[threadIdx.x >> 6] = top;
      __syncthreads();
      for (int w = 0; w < kWavesPerBlock; ++w) top = fmaxf(top, part[w]);
    }
    if (threadIdx.x == 0) {
      int e = 0;
      if (ST == kF16 && top > 0.0f && top <= 3.0e38f) {
        frexpf(top, &e);
        e = 15 - e;      // top 2^e lies in [2^14, 2^15)
        e = e > 120 ? 120 : e;
      }
      a.factor[0] = ldexpf(1.0f, e);
      a.factor[1] = ldexpf(a.scale, -e);
    }
  }
  if (!a.x_rows) return;
  const int64_t chunks = a.x_width / E, all = a.rows * chunks;
  for (int64_t q = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x; q < all;
       q += static_cast<int64_t>(gridDim.x) * kBlock) {
    const int64_t n = q / chunks, c = (q - n * chunks) * E;
    StoredVec<ST, E> v = {};
    if (target_of(a, n) >= 0) {
      if (c + E <= a.K) {
        v = load_vec<ST, E>(a.x, n * a.x_stride + c);
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
          if (c + i < a.K) v[i] = static_cast<const typename Stored<ST>::type*>(a.x)[n * a.x_stride + c + i];
      }
    }
    store_vec<ST, E>(a.x_rows, n * a.x_width + c, v);
  }
}

// Backward: the gradients of a piece's logits, g (2^(exponent - lse) - [target]), zeros
// for rows without a target and past the piece's end.
template <int ST, typename S, int LAYOUT>
__global__ __launch_bounds__(S::threads) void loss_dlogits(LossArgs a, int64_t v0, int64_t piece) {
  __shared__ __align__(1024) unsigned char lds[kLdsBytes<S, LAYOUT>];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wa = (wave % S::NA) * S::WA * 32, wb = (wave / S::NA) * S::WB * 32;
  const int64_t nb = (a.rows + S::TB - 1) / S::TB, na = (piece + S::TA - 1) / S::TA;
  int64_t ta, tb;
  band_order(xcd_contiguous_block(blockIdx.x, gridDim.x), na, nb, &ta, &tb);
  const int64_t a0 = ta * S::TA, b0 = tb * S::TB, left = piece - a0;
  f32x16 acc[S::WA][S::WB];
  const void* x = a.x_rows ? a.x_rows : a.x;
  tile_logits<ST, S, LAYOUT>(a, v0 + a0, left, x, a.x_rows ? a.x_width : a.x_stride, b0, wa, wb, wave,
                             lane, lds, acc);
  const float factor = a.factor[0];
#pragma unroll
  for (int j = 0; j < S::WB; ++j) {
    const int64_t n = b0 + wb + 32 * j + (lane & 31);
    const bool row = n < a.rows;
    const int64_t target = row ? target_of(a, n) : -1;
    const float g = target >= 0 ? a.grad[n] * factor : 0.0f;
    const float lse2 = target >= 0 ? a.lse_in[n] * 1.44269504088896340736f : 0.0f;
    const int64_t at = target - v0 - a0 - wa;
    const bool near = __any(target >= 0 && at >= 0 && at < 32 * S::WA);
    char* p = static_cast<char*>(a.dlogits) +
              (n * a.backward.width + a0 + wa) * StorageTraits<ST>::bytes;
#pragma unroll
    for (int i = 0; i < S::WA; ++i) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        acc[i][j][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][e], a.exponent, -lse2));
      if (near) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (target >= 0 && at == place_of(i, e, lane)) acc[i][j][e] -= 1.0f;
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = target >= 0 ? acc[i][j][e] * g : 0.0f;
      if (left < S::TA) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (wa + place_of(i, e, lane) >= left) acc[i][j][e] = 0.0f;
      }
      const int64_t cols = a.backward.width - a0 - wa - 32 * i;
      if (cols > 0) store_fragment<ST>(p + 32 * i * StorageTraits<ST>::bytes, acc[i][j], cols, row, lane);
    }
  }
}

// A gradient's product of a piece, over one part of the summed index:
//   TABLE  dW[v, k] = sum_n dlogits[n, v] x[n, k],  else  dx[n, k] = sum_v dlogits[n, v] W[v, k].
// Rounded to the output at once where `out` is given, else stored (or added) to the part's sums.
template <int ST, typename S, int LAYOUT, bool TABLE>
__global__ __launch_bounds__(S::threads) void loss_product(LossArgs a, int64_t v0, int64_t piece,
                                                           int64_t splits, int64_t each, void* out,
                                                           int32_t add) {
  __shared__ __align__(1024) unsigned char lds[kLdsBytes<S, LAYOUT>];
  constexpr int bytes = StorageTraits<ST>::bytes, kAhead = kHeldSlices<S, LAYOUT>;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wa = (wave % S::NA) * S::WA * 32, wb = (wave / S::NA) * S::WB * 32;
  const int64_t out_rows = TABLE ? piece : a.rows, whole = TABLE ? a.rows : piece;
  const int64_t na = (a.K + S::TA - 1) / S::TA, nb = (out_rows + S::TB - 1) / S::TB;
  const int64_t q = xcd_contiguous_block(blockIdx.x, gridDim.x);
  const int64_t split = q / (na * nb);
  int64_t ta, tb;
  band_order(q - split * na * nb, na, nb, &ta, &tb);
  const int64_t a0 = ta * S::TA, b0 = tb * S::TB, from = split * each;
  const int64_t depth = whole - from < each ? whole - from : each;
  Operand<ST, false, S::TA, S::NW, LAYOUT, S::RB, kAhead> oa;
  Operand<ST, !TABLE, S::TB, S::NW, LAYOUT, S::RB, kAhead> ob;
  const char* d = static_cast<const char*>(a.dlogits);
  if constexpr (TABLE) {
    // whole chunks: what follows a row's end is zeros
    oa.init(static_cast<const char*>(a.x_rows) + (from * a.x_width + a0) * bytes, a.x_width,
            a.x_width - a0, depth, wave, lane);
    ob.init(d + (from * a.backward.width + b0) * bytes, a.backward.width, a.backward.width - b0, depth,
            wave, lane);
  } else {
    oa.init(static_cast<const char*>(a.table) + ((v0 + from) * a.table_stride + a0) * bytes,
            a.table_stride, a.K - a0, depth, wave, lane);
    constexpr int64_t E = 16 / bytes;  // whole chunks here too
    ob.init(d + (b0 * a.backward.width + from) * bytes, a.backward.width, out_rows - b0,
            (depth + E - 1) / E * E, wave, lane);
  }
  f32x16 acc[S::WA][S::WB];
#pragma unroll
  for (int i = 0; i < S::WA; ++i)
#pragma unroll
    for (int j = 0; j < S::WB; ++j) acc[i][j] = f32x16{};
  accumulate<ST, S, LAYOUT>(oa, ob, depth, lds, wa, wb, wave, lane, acc, [](const u32x4 (&)[S::WB]) {});
  const float undo = out ? a.factor[1] : 1.0f;
  float* parts = (TABLE ? a.dw_parts : a.dx_parts);
#pragma unroll
  for (int i = 0; i < S::WA; ++i) {
    const int64_t c0 = a0 + wa + 32 * i;
    if (c0 >= a.K) continue;
#pragma unroll
    for (int j = 0; j < S::WB; ++j) {
      const int64_t r = b0 + wb + 32 * j + (lane & 31);
      const bool row = r < out_rows;
      if (out) {
        acc[i][j] *= undo;
        char* p = static_cast<char*>(out) + ((TABLE ? v0 + r : r) * a.K + c0) * bytes;
        store_fragment<ST>(p, acc[i][j], a.K - c0, row, lane);
        continue;
      }
      float* p = parts + (split * out_rows + r) * a.K + c0;
      if (add && row) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int c = place_of(0, e, lane);
          if (c0 + c < a.K) acc[i][j][e] += p[c];
        }
      }
      store_fragment<kF32>(p, acc[i][j], a.K - c0, row, lane);
    }
  }
}

// The parts' sums, first part first, to a gradient of n values.
template <int ST>
__global__ __launch_bounds__(kBlock) void loss_sum(LossArgs a, const float* parts, int64_t splits,
                                                   int64_t n, void* out) {
  const int64_t e0 = (static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x) * 4;
  if (e0 >= n) return;
  const float undo = a.factor[1];
  if (e0 + 4 <= n) {
    f32x4 sum = {};
#pragma unroll 8
    for (int64_t s = 0; s < splits; ++s) sum += load_vec<kF32, 4>(parts, s * n + e0);
    StoredVec<ST, 4> v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = static_cast<typename Stored<ST>::type>(sum[j] * undo);
    store_vec<ST, 4>(out, e0, v);
  } else {
    for (int64_t e = e0; e < n; ++e) {
      float sum = 0.0f;
      for (int64_t s = 0; s < splits; ++s) sum += parts[s * n + e];
      store_one<ST>(out, e, sum * undo);
    }
  }
}

using LossLarge = Shape<256, 256, 2, 4, 2, 128>;
using LossMedium = Shape<128, 128, 2, 2, 2, 128>;
using LossSquare = Shape<64, 64, 2, 2, 4, 128>;
using LossNarrow = Shape<128, 32, 4, 1, 4, 128>;

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
  if (tile == 64) return f(LossSquare{});
  f(LossMedium{});
}

template <int ST>
hipError_t launch_loss_forward(const LossArgs& a, hipStream_t s) {
  const auto go = [&](auto shape) {
    using S = decltype(shape);
    const int64_t blocks = ceil_div(a.rows, S::TB) * a.forward.segments;
    with_rows<ST>(a.layout, [&](auto layout) {
      hipLaunchKernelGGL((loss_forward<ST, S, layout>), dim3(static_cast<unsigned>(blocks)),
                         dim3(S::threads), 0, s, a);
    });
  };
  if (a.forward.tile == 32) go(LossNarrow{});
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
  const int64_t n = piece * a.K;
  hipLaunchKernelGGL((loss_sum<ST>), dim3(static_cast<unsigned>(ceil_div(ceil_div(n, 4), kBlock))),
                     dim3(kBlock), 0, s, a, a.dw_parts, splits, n,
                     static_cast<char*>(a.dtable) + v0 * a.K * StorageTraits<ST>::bytes);
  return hipGetLastError();
}

template <int ST>
hipError_t launch_loss_backward(const LossArgs& a, hipStream_t s) {
  constexpr int E = 16 / StorageTraits<ST>::bytes;
  const int64_t chunks = a.x_rows ? a.rows * (a.x_width / E) : 1;
  hipLaunchKernelGGL((loss_prepare<ST>),
                     dim3(static_cast<unsigned>(std::min<int64_t>(ceil_div(chunks, kBlock), 4096))),
                     dim3(kBlock), 0, s, a);
  hipError_t e = hipGetLastError();
  if (a.rows == 0) {  // no rows: a gradient of zeros
    const int64_t all = a.vocab * a.K, most = int64_t{1} << 30;
    for (int64_t v = 0; e == hipSuccess && v < all; v += most) {
      const int64_t n = std::min(most, all - v);
      hipLaunchKernelGGL((loss_sum<ST>), dim3(static_cast<unsigned>(ceil_div(ceil_div(n, 4), kBlock))),
                         dim3(kBlock), 0, s, a, nullptr, int64_t{0}, n,
                         static_cast<char*>(a.dtable) + v * StorageTraits<ST>::bytes);
      e = hipGetLastError();
    }
    return e;
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
  const int64_t n = a.rows * a.K;
  hipLaunchKernelGGL((loss_sum<ST>), dim3(static_cast<unsigned>(ceil_div(ceil_div(n, 4), kBlock))),
                     dim3(kBlock), 0, s, a, a.dx_parts, a.backward.x.splits, n, a.dx);
  return hipGetLastError();
}

template <int ST>
hipError_t launch_loss(const LossArgs& a, bool backward, hipStream_t s) {
  return backward ? launch_loss_backward<ST>(a, s) : launch_loss_forward<ST>(a, s);
}

}  // namespace

#endif  // TBE_LOSS_KERNELS

}  // namespace tbe
