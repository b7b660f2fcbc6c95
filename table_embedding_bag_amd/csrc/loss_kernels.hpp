// loss_kernels.hpp -- the softmax loss's kernels for rows of any width, type and alignment.
//
// A tile's product needs all the registers there are, so what follows it is written to keep
// little across it: targets in 32 bits, rows' information read behind it, branches for what
// is rare, and nothing worked out of the lane's number kept from tile to tile.  What did not fit
// went to memory and back: 16384 rows, 131072 outputs of 512, fp16, forward 2.8 ms, 2.2 without.
#pragma once

#include "products.hpp"
#include "softmax_loss.hpp"
#include "tiles.hpp"

namespace tbe {

namespace {

constexpr float kNegInf = -__builtin_inff();
constexpr int32_t kNegative = 1 << 30;  // of a row's target: its gradient is negative

// What loss_prepare works out of row n.
struct RowInfo {
  float base;
  int32_t target;
  float grad;
};
__device__ __forceinline__ RowInfo row_info(const LossArgs& a, int64_t n) {
  const uint32_t* p = a.row_info + n / 64 * kInfoBlock + n % 64;
  return RowInfo{__uint_as_float(p[0]), static_cast<int32_t>(p[64]), __uint_as_float(p[128])};
}

// The target of row n, or -1 where it has none (or one outside the table).
__device__ __forceinline__ int64_t target_of(const LossArgs& a, int64_t n) {
  const int64_t t = a.index64 ? static_cast<const int64_t*>(a.targets)[n]
                              : static_cast<const int32_t*>(a.targets)[n];
  return t >= 0 && t < a.vocab ? t : -1;
}

// What follows is done where the branch is taken alone: left to itself the compiler may do it
// always and choose afterwards, and keeps what it needs in registers all the time.
__device__ __forceinline__ void rarely() { asm volatile(""); }

// A copy of v that the compiler takes for another value: nothing worked out of it is kept from
// one turn of a loop for the next.
__device__ __forceinline__ int afresh(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Which of the lane's 16 values of a block is row `at` (where real: in 0 .. 31), or -1.
__device__ __forceinline__ int32_t element_of(int32_t at, bool real, int lane) {
  if (!real || (at >> 2 & 1) != lane >> 5) return -1;
  return (at >> 3) * 4 + (at & 3);
}
__device__ __forceinline__ void subtract_at(f32x16& z, int32_t element, float v) {
#pragma unroll
  for (int e = 0; e < 16; ++e) z[e] -= element == e ? v : 0.0f;
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

// Two sums of powers of two relative to a largest exponent each.
__device__ __forceinline__ float2 join_sums(float2 a, float2 b) {
  const float top = fmaxf(a.x, b.x), from = top == kNegInf ? 0.0f : top;
  return make_float2(top, a.y * __builtin_amdgcn_exp2f(a.x - from) + b.y * __builtin_amdgcn_exp2f(b.x - from));
}

// Forward: each row's sum of 2^(exponent - reference) over the segment's tiles, lane by lane;
// joined over lanes and waves once at the end.
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
  float from[S::WB], sum[S::WB];  // what a row's powers are relative to, their sum
  bool unset[S::WB];              // no reference yet
  int32_t target[S::WB];          // tables have at most 2^30 rows
#pragma unroll
  for (int j = 0; j < S::WB; ++j) {
    from[j] = sum[j] = 0.0f;
    unset[j] = true;
    const int64_t n = b0 + wb + 32 * j + (lane & 31);
    target[j] = n < a.rows ? static_cast<int32_t>(target_of(a, n)) : -1;
  }
  for (int64_t t = first; t < last; ++t) {
    const int64_t a0 = t * S::TA, left = a.vocab - a0;
    f32x16 acc[S::WA][S::WB];
    if (t > first) __syncthreads();  // the tile before is read
    tile_logits<ST, S, LAYOUT>(a, a0, left, a.x, a.x_stride, b0, wa, wb, wave, afresh(lane), lds, acc);
    const int place = afresh(lane);
    if (left < S::TA) {  // the last: nothing past the table's end
      rarely();
#pragma unroll
      for (int i = 0; i < S::WA; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (wa + place_of(i, e, place) >= left)
#pragma unroll
            for (int j = 0; j < S::WB; ++j) acc[i][j][e] = kNegInf;
    }
#pragma unroll
    for (int j = 0; j < S::WB; ++j) {
      const int32_t at = target[j] - static_cast<int32_t>(a0) - wa;  // none: below 0
      const bool near = static_cast<uint32_t>(at) < 32u * S::WA;
      if (__any(near)) {
        rarely();
#pragma unroll
        for (int i = 0; i < S::WA; ++i) {
          const int32_t hit = element_of(at - 32 * i, near && at >> 5 == i, place);
          float logit = 0.0f;
#pragma unroll
          for (int e = 0; e < 16; ++e) logit = hit == e ? acc[i][j][e] : logit;
          if (hit >= 0) a.target_logit[b0 + wb + 32 * j + (place & 31)] = logit;
        }
      }
      // The reference is the largest power of the row's first tile (or of the last one whose
      // powers grew past 2^80 of it): no maximum is looked for otherwise, as fp32 holds sums
      // of 2^20 such powers, and what lies far below the reference does not count.
      const auto powers = [&](float reference) {
        float part[4] = {};
#pragma unroll
        for (int i = 0; i < S::WA; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            part[e & 3] += __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][e], a.exponent, -reference));
        return (part[0] + part[1]) + (part[2] + part[3]);
      };
      float now = powers(from[j]);
      const bool again = unset[j] || !(now <= 0x1p80f);  // each lane for itself
      if (__any(again)) {
        rarely();
        float top = kNegInf;
#pragma unroll
        for (int i = 0; i < S::WA; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) top = fmaxf(top, acc[i][j][e]);
        const float next = fmaxf(unset[j] ? kNegInf : from[j], top * a.exponent);
        const bool still = next == kNegInf;
        const float reference = still ? 0.0f : next, other = powers(reference);
        if (again) {
          now = other;
          sum[j] = unset[j] ? sum[j] : sum[j] * __builtin_amdgcn_exp2f(from[j] - reference);
          from[j] = reference;
          unset[j] = still;
        }
      }
      sum[j] += now;
    }
  }
  // the two halves of a wave, then the waves that have the same rows
  __syncthreads();
  float2* joined = reinterpret_cast<float2*>(lds);
#pragma unroll
  for (int j = 0; j < S::WB; ++j) {
    const float2 mine = make_float2(unset[j] ? kNegInf : from[j], sum[j]);
    const float2 other = make_float2(__shfl_xor(mine.x, 32), __shfl_xor(mine.y, 32));
    const float2 both = join_sums(mine, other);
    if (lane < 32) joined[(wave % S::NA) * S::TB + wb + 32 * j + lane] = both;
  }
  __syncthreads();
  for (int r = threadIdx.x; r < S::TB; r += S::threads) {
    if (b0 + r >= a.rows) break;
    float2 v = joined[r];
#pragma unroll
    for (int w = 1; w < S::NA; ++w) v = join_sums(v, joined[w * S::TB + r]);
    a.parts[segment * a.rows + b0 + r] = v;
  }
}

// A row's segments joined, 16 rows a workgroup, 16 segments at a time.
template <int ST>
__global__ __launch_bounds__(kBlock) void loss_join(LossArgs a) {
  __shared__ float2 part[16][16];
  const int r = threadIdx.x & 15, slice = threadIdx.x >> 4;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 16 + r;
  float2 sum = make_float2(kNegInf, 0.0f);
  if (n < a.rows)
#pragma unroll 4
    for (int64_t g = slice; g < a.forward.segments; g += 16) sum = join_sums(sum, a.parts[g * a.rows + n]);
  part[slice][r] = sum;
  __syncthreads();
  if (slice == 0 && n < a.rows) {
    for (int i = 1; i < 16; ++i) sum = join_sums(sum, part[i][r]);
    // in 64 bits: the difference of two large values is what is asked for
    const double ln2 = 0.69314718055994530942;
    const double power = ln2 * (static_cast<double>(sum.x) + static_cast<double>(log2f(sum.y)));
    a.lse[n] = static_cast<float>(power);
    a.loss[n] = target_of(a, n) < 0 ? 0.0f
                                    : static_cast<float>(power - ln2 * static_cast<double>(a.exponent) *
                                                                     static_cast<double>(a.target_logit[n]));
  }
}

// fp16 gradients of the logits are multiplied by 2^14 over the largest row gradient's power
// of two, so that probabilities down to 2^-28 of it stay normal numbers: that factor, what
// undoes it times the scale, and its exponent.
__global__ __launch_bounds__(1024) void loss_factor(LossArgs a) {
  __shared__ float part[16];
  float top = 0.0f;
#pragma unroll 4
  for (int64_t n = threadIdx.x; n < a.rows; n += 1024)
    top = fmaxf(top, target_of(a, n) >= 0 ? fabsf(a.grad[n]) : 0.0f);
  for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
  if (lane_id() == 0) part[threadIdx.x >> 6] = top;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 0; w < 16; ++w) top = fmaxf(top, part[w]);
  int e = 0;
  if (top > 0.0f && top <= 3.0e38f) {
    frexpf(top, &e);
    e = 15 - e;  // top 2^e lies in [2^14, 2^15)
    e = e > 120 ? 120 : e;
  }
  a.factor[0] = ldexpf(1.0f, e);
  a.factor[1] = ldexpf(a.scale, -e);
  a.factor[2] = static_cast<float>(e);
}

// x for the gradients' products: rows without a target are zeros, whatever they hold, and
// so is what follows a row's end.
// row_info gets what a row's powers are relative to, log2(e^lse / |g factor|),
// +infinity where there is no target (powers of 0), its target, -1 for none, with a bit
// set where g is negative, and g times the factor.
template <int ST>
__global__ __launch_bounds__(kBlock) void loss_prepare(LossArgs a) {
  constexpr int E = 16 / StorageTraits<ST>::bytes;
  const int32_t e = ST == kF16 ? static_cast<int32_t>(a.factor[2]) : 0;
  if (ST != kF16 && blockIdx.x == 0 && threadIdx.x == 0) {
    a.factor[0] = 1.0f;
    a.factor[1] = a.scale;
  }
  const int64_t padded = (a.rows + 63) / 64 * 64;
  for (int64_t n = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x; n < padded;
       n += static_cast<int64_t>(gridDim.x) * kBlock) {
    const int64_t target = n < a.rows ? target_of(a, n) : -1;
    float base = __builtin_inff(), scaled = 0.0f;
    int32_t word = -1;
    if (target >= 0) {
      const float g = a.grad[n];
      // in 64 bits: the difference is what powers of two are taken of
      base = static_cast<float>(static_cast<double>(a.lse_in[n]) * 1.44269504088896340736 -
                                static_cast<double>(log2f(fabsf(g))) - e);
      word = static_cast<int32_t>(target) | (g < 0.0f ? kNegative : 0);
      scaled = ldexpf(g, e);
    }
    uint32_t* info = a.row_info + n / 64 * kInfoBlock + n % 64;
    info[0] = __float_as_uint(base);
    info[64] = static_cast<uint32_t>(word);
    info[128] = __float_as_uint(scaled);
  }
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
  tile_logits<ST, S, LAYOUT>(a, v0 + a0, left, a.x_rows, a.x_width, b0, wa, wb, wave, lane, lds, acc);
#pragma unroll
  for (int j = 0; j < S::WB; ++j) {
    const int64_t n = b0 + wb + 32 * j + (lane & 31);
    const bool row = n < a.rows;
    const RowInfo info = row ? row_info(a, n) : RowInfo{__builtin_inff(), -1, 0.0f};
    const bool negative = info.target >= 0 && (info.target & kNegative);
    const int32_t at = (info.target & ~kNegative) - static_cast<int32_t>(v0 + a0) - wa;
    const bool near = info.target >= 0 && static_cast<uint32_t>(at) < 32u * S::WA;
    const bool any_near = __any(near), turned = __any(negative);
    // 2-byte values: powers times |g| at once.  fp32 would tell that the exponent's rounding
    // grows with log2 |g|.
    const float g = fabsf(info.grad);
    const float base = ST == kF32 ? (info.target >= 0 ? a.lse_in[n] * 1.44269504088896340736f : __builtin_inff())
                                  : info.base;
    char* p = static_cast<char*>(a.dlogits) +
              (n * a.backward.width + a0 + wa) * StorageTraits<ST>::bytes;
#pragma unroll
    for (int i = 0; i < S::WA; ++i) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        acc[i][j][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][e], a.exponent, -base));
      if (any_near) {
        rarely();
        subtract_at(acc[i][j], element_of(at - 32 * i, near && at >> 5 == i, lane), ST == kF32 ? 1.0f : g);
      }
      if constexpr (ST == kF32) {
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] *= g;
      }
      if (turned) {
        rarely();
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = negative ? -acc[i][j][e] : acc[i][j][e];
      }
      if (left < S::TA) {
        rarely();
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

}  // namespace
}  // namespace tbe
