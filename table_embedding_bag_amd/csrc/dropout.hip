// dropout.hip -- dropout whose mask is computed, never stored.
//
// Element n of the row-major [rows, cols] matrix takes word n % 4 of the
// 7-round Philox4x32 block (Salmon, Moraes, Dror, Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", SC'11) of counter offset + n / 4 under the
// 64-bit key `seed`; it is kept where that word is at least floor(p 2^32).
// The gradient's map is the same one, so the backward pass recomputes the
// mask from (seed, offset).
//
// One pass: every element read and written once.  A block costs 14 32 x 32 ->
// 64 bit products for four elements.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "layers.hpp"

using namespace tbe;

namespace {

constexpr int kRounds = 7;
constexpr uint32_t kMul0 = 0xD2511F53u, kMul1 = 0xCD9E8D57u;    // multipliers
constexpr uint32_t kWeyl0 = 0x9E3779B9u, kWeyl1 = 0xBB67AE85u;  // key increments

struct DropoutArgs {
  const void* x;
  const void* residual;  // null: none
  void* y;
  int64_t x_stride, r_stride, y_stride;  // elements between rows
  int64_t n, cols;                       // n = rows * cols
  uint64_t inverse;                      // ceil(2^64 / cols) (0 for cols = 1)
  uint64_t seed, offset;
  uint32_t least;                        // smallest word that is kept
  int32_t none;                          // p = 1: nothing is kept
  float scale;                           // 1 / (1 - p)
};

__device__ __forceinline__ uint4 philox(uint64_t counter, uint64_t seed) {
  uint32_t c0 = static_cast<uint32_t>(counter), c1 = static_cast<uint32_t>(counter >> 32);
  uint32_t c2 = 0u, c3 = 0u;
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const uint64_t p0 = static_cast<uint64_t>(c0) * kMul0, p1 = static_cast<uint64_t>(c2) * kMul1;
    c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ k0;
    c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ k1;
    c1 = static_cast<uint32_t>(p1);
    c3 = static_cast<uint32_t>(p0);
    k0 += kWeyl0;
    k1 += kWeyl1;
  }
  return make_uint4(c0, c1, c2, c3);
}

// A thread takes a group of E elements (16 bytes); groups start at multiples of E
// in the packed numbering, so that they are whole Philox blocks whatever the row
// length.  PACKED: all rows lie end to end, element n is at n.  One group a thread:
// four, their loads in flight together, were slower at every size (2048 x 128 fp32
// 3.0 -> 3.8 us, 32768 x 4096 bf16 with a residual 143 -> 151 and its gradient 93 ->
// 103, kernel times).  Both directions of the latter take 227 us a pass, 5.9 TB/s, more
// than a copy's 5.2: memory bounds it.
template <int ST, bool RESIDUAL, bool PACKED>
__global__ __launch_bounds__(kBlock) void dropout_map(DropoutArgs a) {
  constexpr int E = 16 / StorageTraits<ST>::bytes;
  const int64_t groups = (a.n + E - 1) / E, step = static_cast<int64_t>(gridDim.x) * kBlock;
  for (int64_t g = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x; g < groups; g += step) {
    const int64_t n0 = g * E;
    int64_t row = 0, col = n0;
    bool whole = n0 + E <= a.n;  // the group's E elements lie in one row
    if constexpr (!PACKED) {
      // n0 / cols: the reciprocal's quotient is at most one too large
      int64_t q = a.inverse ? static_cast<int64_t>(__umul64hi(static_cast<uint64_t>(n0), a.inverse))
                            : n0;
      if (q * a.cols > n0) --q;
      row = q;
      col = n0 - q * a.cols;
      whole = whole && col + E <= a.cols;
    }
    StoredVec<ST, E> v, res;
    if (whole) {
      v = load_vec<ST, E>(a.x, row * a.x_stride + col);
      if constexpr (RESIDUAL) res = load_vec<ST, E>(a.residual, row * a.r_stride + col);
    }
    uint32_t w[E];
#pragma unroll
    for (int b = 0; b < E / 4; ++b) {
      const uint4 p = philox(a.offset + static_cast<uint64_t>(g * (E / 4) + b), a.seed);
      w[4 * b] = p.x, w[4 * b + 1] = p.y, w[4 * b + 2] = p.z, w[4 * b + 3] = p.w;
    }
    if (whole) {
      StoredVec<ST, E> out;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const bool kept = w[i] >= a.least && !a.none;
        float f = kept ? static_cast<float>(v[i]) * a.scale : 0.0f;
        if constexpr (RESIDUAL) f += static_cast<float>(res[i]);
        out[i] = static_cast<typename Stored<ST>::type>(f);
      }
      store_vec<ST, E>(a.y, row * a.y_stride + col, out);
    } else {  // the matrix's last elements, or a group that runs over a row's end
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (n0 + i >= a.n) break;
        const bool kept = w[i] >= a.least && !a.none;
        float f = kept ? load_one<ST>(a.x, row * a.x_stride + col) * a.scale : 0.0f;
        if constexpr (RESIDUAL) f += load_one<ST>(a.residual, row * a.r_stride + col);
        store_one<ST>(a.y, row * a.y_stride + col, f);
        if (++col == a.cols) col = 0, ++row;
      }
    }
  }
}

template <int ST, bool RESIDUAL, bool PACKED>
hipError_t launch_dropout(const DropoutArgs& a, hipStream_t s) {
  constexpr int E = 16 / StorageTraits<ST>::bytes;
  const int64_t groups = (a.n + E - 1) / E;
  // at most 2^31 threads in a launch
  const int64_t blocks = std::min<int64_t>((groups + kBlock - 1) / kBlock, (int64_t{1} << 31) / kBlock);
  hipLaunchKernelGGL((dropout_map<ST, RESIDUAL, PACKED>), dim3(static_cast<unsigned>(blocks)),
                     dim3(kBlock), 0, s, a);
  return hipGetLastError();
}

template <int ST>
hipError_t launch_dropout(const DropoutArgs& a, bool packed, hipStream_t s) {
  if (a.residual)
    return packed ? launch_dropout<ST, true, true>(a, s) : launch_dropout<ST, true, false>(a, s);
  return packed ? launch_dropout<ST, false, true>(a, s) : launch_dropout<ST, false, false>(a, s);
}

}  // namespace

extern "C" tbe_status tbe_dropout(const void* x, int64_t x_stride, const void* residual,
                                  int64_t residual_stride, void* y, int64_t y_stride, int64_t rows,
                                  int64_t cols, int32_t dtype, double p, uint64_t seed,
                                  uint64_t offset, void* stream) {
  if (rows < 0 || cols < 0 || !known_dtype(dtype)) return TBE_ERR_INVALID_ARGUMENT;
  if (!(p >= 0.0 && p <= 1.0)) return TBE_ERR_INVALID_ARGUMENT;  // NaN too
  if (rows == 0 || cols == 0) return TBE_OK;
  if (!x || !y) return TBE_ERR_INVALID_ARGUMENT;
  if (rows > 1 && (x_stride < 0 || y_stride < cols || (residual && residual_stride < 0)))
    return TBE_ERR_INVALID_ARGUMENT;
  const size_t e = dtype_bytes(dtype);
  if (!aligned_to(x, e) || !aligned_to(y, e) || (residual && !aligned_to(residual, e)))
    return TBE_ERR_INVALID_ARGUMENT;
  if (rows > (int64_t{1} << 35) / cols) return TBE_ERR_UNSUPPORTED;
  DropoutArgs a{};
  a.x = x;
  a.residual = residual;
  a.y = y;
  a.x_stride = x_stride;
  a.r_stride = residual_stride;
  a.y_stride = y_stride;
  a.n = rows * cols;
  a.cols = cols;
  a.inverse = cols == 1 ? 0 : ~uint64_t{0} / static_cast<uint64_t>(cols) + 1;
  a.seed = seed;
  a.offset = offset;
  a.none = p == 1.0;
  a.least = a.none ? 0u : static_cast<uint32_t>(std::floor(p * 4294967296.0));
  a.scale = a.none ? 0.0f : static_cast<float>(1.0 / (1.0 - p));
  const bool packed = rows == 1 || (x_stride == cols && y_stride == cols &&
                                    (!residual || residual_stride == cols));
  hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t err = dtype == TBE_F32   ? launch_dropout<kF32>(a, packed, s)
                         : dtype == TBE_F16 ? launch_dropout<kF16>(a, packed, s)
                                            : launch_dropout<kBF16>(a, packed, s);
  return err == hipSuccess ? TBE_OK : TBE_ERR_HIP;
}
