// norm.hip -- layer norm over rows and its gradients:
//   m = mean(x), r = 1 / sqrt(mean((x - m)^2) + eps), n = (x - m) r, y = n w + b;
//   dx = r (gw - mean(gw) - n mean(gw n)) with gw = g w,  dw = sum_rows g n,  db = sum_rows g.
// The squares are summed after the mean is subtracted, in fp32.
//
// Memory bounds both passes: a row's values stay in registers between its sums and its
// outputs, and the next row's are on their way meanwhile.  32768 x 4096 bf16, one call after
// the other: forward 96 us (5.6 TB/s), backward 160 us (5.0 TB/s; about 190 with the weight read for
// every row, 250 without the next row's loads) and its join 8; under the profiler, between other
// kernels, 86 to 94 and 163 to 195.  The gradients over the rows are summed by each workgroup
// for its rows, at most 512 in a row in fp32, then over the workgroups in 64 bits, in a fixed order:
// their rounding does not grow with the rows.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "layers.hpp"

using namespace tbe;

namespace {

struct NormArgs {
  const void* x;
  const void* weight;  // or null: ones
  const void* bias;    // or null: zeros
  void* y;
  float2* stats;       // [rows] {m, r}, or null
  const float2* stats_in;
  const void* grad;
  void* dx;            // or null
  void* dweight;       // or null
  void* dbias;         // or null
  float* parts;        // [blocks][2][cols]: sums of g n and of g
  int64_t x_stride, y_stride, g_stride, dx_stride;
  int64_t rows, cols;
  int64_t blocks;      // of the backward pass
  float eps, count;    // count: cols (divided by: the mean of equal values is that value)
};

// Neighbours, pairs, quads, halves of 16 lanes, 16 and 32 lanes change places: both sides of
// every step add the same two values, and no step goes through LDS.
template <int CTRL>
__device__ __forceinline__ float swap_lanes(float v) {
  const uint32_t u = __float_as_uint(v);
  return __uint_as_float(__builtin_amdgcn_update_dpp(u, u, CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float wave_sum(float v) {
  v += swap_lanes<0xB1>(v);
  v += swap_lanes<0x4E>(v);
  v += swap_lanes<0x141>(v);
  v += swap_lanes<0x140>(v);
  const uint32_t u = __float_as_uint(v);
  const auto rows = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  v = __uint_as_float(rows[0]) + __uint_as_float(rows[1]);
  const uint32_t w = __float_as_uint(v);
  const auto halves = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return __uint_as_float(halves[0]) + __uint_as_float(halves[1]);
}

// The sum over a row's threads: a wave (NW = 1) or a workgroup of NW waves.  `scratch`
// alternates between two buffers: one barrier a sum.
template <int NW>
__device__ __forceinline__ float2 row_sum(float2 v, float2 (*scratch)[NW], int* turn) {
  v = make_float2(wave_sum(v.x), wave_sum(v.y));
  if constexpr (NW == 1) return v;
  float2* const at = scratch[*turn];
  *turn ^= 1;
  if (lane_id() == 0) at[threadIdx.x >> 6] = v;
  __syncthreads();
  float2 s = at[0];
#pragma unroll
  for (int w = 1; w < NW; ++w) s.x += at[w].x, s.y += at[w].y;
  return s;
}
template <int NW>
__device__ __forceinline__ float row_sum(float v, float2 (*scratch)[NW], int* turn) {
  if constexpr (NW == 1) return wave_sum(v);
  return row_sum<NW>(make_float2(v, 0.0f), scratch, turn).x;
}

// E values from element c of a row of `cols`; zeros past its end.
template <int ST, int E>
__device__ __forceinline__ StoredVec<ST, E> load_stored(const void* base, int64_t at, int64_t c, int64_t cols) {
  StoredVec<ST, E> v = {};
  if (c + E <= cols) {
    v = load_vec<ST, E>(base, at + c);
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (c + i < cols) v[i] = static_cast<const typename Stored<ST>::type*>(base)[at + c + i];
  }
  return v;
}
template <int ST, int E>
__device__ __forceinline__ void store_part(void* base, int64_t at, int64_t c, int64_t cols, const float* f) {
  if (c + E <= cols) {
    StoredVec<ST, E> v;
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = static_cast<typename Stored<ST>::type>(f[i]);
    store_vec<ST, E>(base, at + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (c + i < cols) store_one<ST>(base, at + c + i, f[i]);
  }
}

// A row by NW waves, each thread C chunks of 16 bytes that stay in registers.
template <int ST, int NW, int C>
__global__ __launch_bounds__(NW == 1 ? kBlock : NW * 64) void norm_forward(NormArgs a) {
  constexpr int E = 16 / StorageTraits<ST>::bytes, T = NW * 64;
  __shared__ float2 scratch[2][NW];
  int turn = 0;
  constexpr int R = NW == 1 ? kWavesPerBlock : 1;  // rows at a time
  const int t = NW == 1 ? lane_id() : threadIdx.x, mine = NW == 1 ? threadIdx.x >> 6 : 0;
  // a row's values are on their way while the row before is worked on
  StoredVec<ST, E> next[C];
  const auto fetch = [&](int64_t row) {
#pragma unroll
    for (int k = 0; k < C; ++k) next[k] = load_stored<ST, E>(a.x, row * a.x_stride, (k * T + t) * E, a.cols);
  };
  const int64_t first = static_cast<int64_t>(blockIdx.x) * R + mine, step = static_cast<int64_t>(gridDim.x) * R;
  if (first < a.rows) fetch(first);
  StoredVec<ST, E> w[C], b[C];
#pragma unroll
  for (int k = 0; k < C; ++k) {
    if (a.weight) w[k] = load_stored<ST, E>(a.weight, 0, (k * T + t) * E, a.cols);
    if (a.bias) b[k] = load_stored<ST, E>(a.bias, 0, (k * T + t) * E, a.cols);
  }
  for (int64_t row = first; row < a.rows; row += step) {
    float f[C][E];
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < C; ++k)
#pragma unroll
      for (int i = 0; i < E; ++i) {
        f[k][i] = static_cast<float>(next[k][i]);
        sum += f[k][i];
      }
    if (row + step < a.rows) fetch(row + step);
    const float m = row_sum<NW>(sum, scratch, &turn) / a.count;
    float squares = 0.0f;
#pragma unroll
    for (int k = 0; k < C; ++k)
#pragma unroll
      for (int i = 0; i < E; ++i) {
        f[k][i] = (k * T + t) * E + i < a.cols ? f[k][i] - m : 0.0f;
        squares += f[k][i] * f[k][i];
      }
    const float r = 1.0f / sqrtf(row_sum<NW>(squares, scratch, &turn) / a.count + a.eps);
    if (a.stats && t == 0) a.stats[row] = make_float2(m, r);
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const int64_t c = (k * T + t) * E;
      if (c >= a.cols) continue;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        f[k][i] *= r;
        if (a.weight) f[k][i] *= static_cast<float>(w[k][i]);
        if (a.bias) f[k][i] += static_cast<float>(b[k][i]);
      }
      store_part<ST, E>(a.y, row * a.y_stride, c, a.cols, f[k]);
    }
  }
}

// Rows blockIdx.x, blockIdx.x + blocks, ...: their dx, and this workgroup's sums for the
// weight's and the bias's gradients.
template <int ST, int NW, int C>
__global__ __launch_bounds__(NW == 1 ? kBlock : NW * 64) void norm_backward(NormArgs a) {
  constexpr int E = 16 / StorageTraits<ST>::bytes, T = NW * 64;
  constexpr int R = NW == 1 ? kWavesPerBlock : 1;  // rows at a time
  __shared__ float2 scratch[2][NW];
  int turn = 0;
  __shared__ float shared[R > 1 ? R * T * E * C : 1];
  const int t = NW == 1 ? lane_id() : threadIdx.x, mine = NW == 1 ? threadIdx.x >> 6 : 0;
  float gn[C][E] = {}, gs[C][E] = {};
  // a row's values are on their way while the row before is worked on
  StoredVec<ST, E> x_next[C], g_next[C];
  const auto fetch = [&](int64_t row) {
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const int64_t c = (k * T + t) * E;
      x_next[k] = load_stored<ST, E>(a.x, row * a.x_stride, c, a.cols);
      g_next[k] = load_stored<ST, E>(a.grad, row * a.g_stride, c, a.cols);
    }
  };
  const int64_t first = static_cast<int64_t>(blockIdx.x) * R + mine, step = a.blocks * R;
  if (first < a.rows) fetch(first);
  StoredVec<ST, E> w[C];
#pragma unroll
  for (int k = 0; k < C; ++k)
    if (a.weight) w[k] = load_stored<ST, E>(a.weight, 0, (k * T + t) * E, a.cols);
  for (int64_t row = first; row < a.rows; row += step) {
    const float2 st = a.stats_in[row];
    float n[C][E], g[C][E];
    float2 sums = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < C; ++k)
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const bool inside = (k * T + t) * E + i < a.cols;
        g[k][i] = static_cast<float>(g_next[k][i]);
        n[k][i] = (static_cast<float>(x_next[k][i]) - st.x) * st.y;
        gn[k][i] += inside ? g[k][i] * n[k][i] : 0.0f;
        gs[k][i] += g[k][i];
      }
    if (row + step < a.rows) fetch(row + step);
    if (!a.dx) continue;
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const int64_t c = (k * T + t) * E;
      if (a.weight)
#pragma unroll
        for (int i = 0; i < E; ++i) g[k][i] *= static_cast<float>(w[k][i]);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        sums.x += g[k][i];
        sums.y += c + i < a.cols ? g[k][i] * n[k][i] : 0.0f;
      }
    }
    sums = row_sum<NW>(sums, scratch, &turn);
    const float s1 = sums.x / a.count, s2 = sums.y / a.count;
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const int64_t c = (k * T + t) * E;
      if (c >= a.cols) continue;
#pragma unroll
      for (int i = 0; i < E; ++i) g[k][i] = st.y * (g[k][i] - s1 - n[k][i] * s2);
      store_part<ST, E>(a.dx, row * a.dx_stride, c, a.cols, g[k]);
    }
  }
  if (!a.parts) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (which == 0 ? !a.dweight : !a.dbias) continue;
    float* out = a.parts + (2 * static_cast<int64_t>(blockIdx.x) + which) * a.cols;
    if constexpr (R > 1) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < C; ++k)
#pragma unroll
        for (int i = 0; i < E; ++i)
          shared[(mine * C + k) * T * E + t * E + i] = which == 0 ? gn[k][i] : gs[k][i];
      __syncthreads();
      for (int64_t c = threadIdx.x; c < a.cols; c += kBlock) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < R; ++w) s += shared[w * C * T * E + c];
        out[c] = s;
      }
    } else {
#pragma unroll
      for (int k = 0; k < C; ++k)
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const int64_t c = (k * T + t) * E + i;
          if (c < a.cols) out[c] = which == 0 ? gn[k][i] : gs[k][i];
        }
    }
  }
}

// Rows too long for registers: read again for every use.
template <int ST>
__global__ __launch_bounds__(1024) void norm_forward_long(NormArgs a) {
  constexpr int NW = 16;
  __shared__ float2 scratch[2][NW];
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const int64_t at = row * a.x_stride;
    float sum = 0.0f;
    for (int64_t c = threadIdx.x; c < a.cols; c += NW * 64) sum += load_one<ST>(a.x, at + c);
    const float m = row_sum<NW>(sum, scratch, &turn) / a.count;
    float squares = 0.0f;
    for (int64_t c = threadIdx.x; c < a.cols; c += NW * 64) {
      const float d = load_one<ST>(a.x, at + c) - m;
      squares += d * d;
    }
    const float r = 1.0f / sqrtf(row_sum<NW>(squares, scratch, &turn) / a.count + a.eps);
    if (a.stats && threadIdx.x == 0) a.stats[row] = make_float2(m, r);
    for (int64_t c = threadIdx.x; c < a.cols; c += NW * 64) {
      float v = (load_one<ST>(a.x, at + c) - m) * r;
      if (a.weight) v *= load_one<ST>(a.weight, c);
      if (a.bias) v += load_one<ST>(a.bias, c);
      store_one<ST>(a.y, row * a.y_stride + c, v);
    }
  }
}
template <int ST>
__global__ __launch_bounds__(1024) void norm_backward_long(NormArgs a) {
  constexpr int NW = 16;
  __shared__ float2 scratch[2][NW];
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const int64_t at = row * a.x_stride, g_at = row * a.g_stride;
    const float2 st = a.stats_in[row];
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t c = threadIdx.x; c < a.cols; c += NW * 64) {
      float g = load_one<ST>(a.grad, g_at + c);
      if (a.weight) g *= load_one<ST>(a.weight, c);
      s1 += g;
      s2 += g * (load_one<ST>(a.x, at + c) - st.x) * st.y;
    }
    s1 = row_sum<NW>(s1, scratch, &turn) / a.count;
    s2 = row_sum<NW>(s2, scratch, &turn) / a.count;
    for (int64_t c = threadIdx.x; c < a.cols; c += NW * 64) {
      float g = load_one<ST>(a.grad, g_at + c);
      if (a.weight) g *= load_one<ST>(a.weight, c);
      const float n = (load_one<ST>(a.x, at + c) - st.x) * st.y;
      store_one<ST>(a.dx, row * a.dx_stride + c, st.y * (g - s1 - n * s2));
    }
  }
}
// ... and the workgroups' sums for the gradients over the rows, 64 columns a workgroup.
template <int ST>
__global__ __launch_bounds__(kBlock) void norm_sums_long(NormArgs a) {
  __shared__ float part[2][kWavesPerBlock][64];
  const int lane = lane_id(), w = threadIdx.x >> 6;
  const int64_t c = static_cast<int64_t>(blockIdx.y) * 64 + lane;
  float gn = 0.0f, gs = 0.0f;
  if (c < a.cols)
    for (int64_t n = static_cast<int64_t>(blockIdx.x) * kWavesPerBlock + w; n < a.rows;
         n += a.blocks * kWavesPerBlock) {
      const float2 st = a.stats_in[n];
      const float g = load_one<ST>(a.grad, n * a.g_stride + c);
      gn += g * (load_one<ST>(a.x, n * a.x_stride + c) - st.x) * st.y;
      gs += g;
    }
  part[0][w][lane] = gn;
  part[1][w][lane] = gs;
  __syncthreads();
  if (w < 2 && c < a.cols) {
    float s = 0.0f;
    for (int i = 0; i < kWavesPerBlock; ++i) s += part[w][i][lane];
    a.parts[(2 * static_cast<int64_t>(blockIdx.x) + w) * a.cols + c] = s;
  }
}

// The workgroups' sums to the gradients, 16 columns a workgroup, 64 of them at a time; in 64 bits,
// as there may be many.
template <int ST>
__global__ __launch_bounds__(1024) void norm_join(NormArgs a) {
  __shared__ double part[64][16];
  const int column = threadIdx.x & 15, w = threadIdx.x >> 4, which = blockIdx.y;
  void* out = which == 0 ? a.dweight : a.dbias;
  if (!out) return;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 16 + column;
  double s = 0.0;
  if (c < a.cols)
#pragma unroll 8
    for (int64_t b = w; b < a.blocks; b += 64) s += a.parts[(2 * b + which) * a.cols + c];
  part[w][column] = s;
  __syncthreads();
  if (w == 0 && c < a.cols) {
    s = 0.0;
    for (int i = 0; i < 64; ++i) s += part[i][column];
    store_one<ST>(out, c, static_cast<float>(s));
  }
}

constexpr int64_t kMaxRows = int64_t{1} << 30;
constexpr int64_t kMaxCols = int64_t{1} << 20;
// Workgroups; each takes every so many-th row.  32768 x 4096 bf16: the forward pass 96 us
// with 8192 of them, 105 with 1024, 92 to 100 with one a row; the backward pass, which has as
// many sums to join, 168 with 512 (and the join), 183 with 1024, 238 with 256.
constexpr int64_t kMaxGrid = 8192, kBackwardGrid = 512;
constexpr int64_t kMaxTerms = 512;  // of a workgroup's sums over its rows: beyond, more workgroups

dim3 grid_of(int64_t blocks) { return dim3(static_cast<unsigned>(std::min(blocks, kMaxGrid))); }

int64_t backward_blocks(int64_t rows, int64_t cols, int32_t dtype) {
  const int64_t e = 16 / dtype_bytes(dtype);
  const int64_t each = cols <= 128 * e ? kWavesPerBlock : 1;  // rows of a workgroup at a time
  const int64_t steps = (rows + each - 1) / each;
  return std::max(std::max<int64_t>(1, std::min(steps, kBackwardGrid)), (steps + kMaxTerms - 1) / kMaxTerms);
}

size_t parts_bytes(int64_t rows, int64_t cols, int32_t dtype) {
  return static_cast<size_t>(backward_blocks(rows, cols, dtype)) * 2 * cols * sizeof(float);
}

// f(waves of a row, chunks of a thread), 0 waves for rows that are too long
template <int ST, typename F>
void with_shape(int64_t cols, F f) {
  constexpr int E = 16 / StorageTraits<ST>::bytes;
  const auto i = [](auto n) { return n; };
  using std::integral_constant;
  const int64_t chunks = (cols + E - 1) / E;
  if (chunks <= 64) return f(i(integral_constant<int, 1>{}), i(integral_constant<int, 1>{}));
  if (chunks <= 128) return f(i(integral_constant<int, 1>{}), i(integral_constant<int, 2>{}));
  if (chunks <= 256) return f(i(integral_constant<int, 4>{}), i(integral_constant<int, 1>{}));
  if (chunks <= 512) return f(i(integral_constant<int, 4>{}), i(integral_constant<int, 2>{}));
  if (chunks <= 1024) return f(i(integral_constant<int, 8>{}), i(integral_constant<int, 2>{}));
  if (chunks <= 2048) return f(i(integral_constant<int, 16>{}), i(integral_constant<int, 2>{}));
  f(i(integral_constant<int, 0>{}), i(integral_constant<int, 0>{}));
}

template <int ST>
hipError_t launch_forward(const NormArgs& a, hipStream_t s) {
  const auto go = [&](auto nw, auto c) {
    constexpr int NW = nw, C = c;
    if constexpr (NW == 0)
      hipLaunchKernelGGL((norm_forward_long<ST>), grid_of(a.rows), dim3(1024), 0, s, a);
    else
      hipLaunchKernelGGL((norm_forward<ST, NW, C>),
                         grid_of(NW == 1 ? (a.rows + kWavesPerBlock - 1) / kWavesPerBlock : a.rows),
                         dim3(NW == 1 ? kBlock : NW * 64), 0, s, a);
  };
  with_shape<ST>(a.cols, go);
  return hipGetLastError();
}

template <int ST>
hipError_t launch_backward(const NormArgs& a, hipStream_t s) {
  const unsigned columns = static_cast<unsigned>((a.cols + 63) / 64);
  if (a.rows > 0)
    with_shape<ST>(a.cols, [&](auto nw, auto c) {
      constexpr int NW = nw, C = c;
      const unsigned blocks = static_cast<unsigned>(a.blocks);
      if constexpr (NW == 0) {
        // the sums first: dx may lie where the gradient does
        if (a.parts)
          hipLaunchKernelGGL((norm_sums_long<ST>), dim3(blocks, columns), dim3(kBlock), 0, s, a);
        if (a.dx)
          hipLaunchKernelGGL((norm_backward_long<ST>), grid_of(a.rows), dim3(1024), 0, s, a);
      } else {
        hipLaunchKernelGGL((norm_backward<ST, NW, C>), dim3(blocks), dim3(NW == 1 ? kBlock : NW * 64), 0, s,
                           a);
      }
    });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || (!a.dweight && !a.dbias)) return e;
  hipLaunchKernelGGL((norm_join<ST>), dim3(static_cast<unsigned>((a.cols + 15) / 16), 2), dim3(1024), 0, s, a);
  return hipGetLastError();
}

tbe_status check_sizes(int64_t rows, int64_t cols, int32_t dtype) {
  if (rows < 0 || cols < 1 || !known_dtype(dtype)) return TBE_ERR_INVALID_ARGUMENT;
  if (rows > kMaxRows || cols > kMaxCols) return TBE_ERR_UNSUPPORTED;
  return TBE_OK;
}

}  // namespace

extern "C" {

tbe_status tbe_layer_norm_sizes(int64_t rows, int64_t cols, int32_t dtype, size_t* backward_bytes) {
  if (!backward_bytes) return TBE_ERR_INVALID_ARGUMENT;
  const tbe_status st = check_sizes(rows, cols, dtype);
  if (st == TBE_OK) *backward_bytes = parts_bytes(rows, cols, dtype);
  return st;
}

tbe_status tbe_layer_norm(const void* x, int64_t x_stride, const void* weight, const void* bias, void* y,
                          int64_t y_stride, float* stats, int64_t rows, int64_t cols, int32_t dtype,
                          double eps, void* stream) {
  const tbe_status st = check_sizes(rows, cols, dtype);
  if (st != TBE_OK) return st;
  if (!(eps >= 0.0 && eps <= 1e30)) return TBE_ERR_INVALID_ARGUMENT;  // NaN too
  if (rows == 0) return TBE_OK;
  const size_t e = dtype_bytes(dtype);
  if (!x || !y || !aligned_to(x, e) || !aligned_to(weight, e) || !aligned_to(bias, e) || !aligned_to(y, e) ||
      !aligned_to(stats, 8))
    return TBE_ERR_INVALID_ARGUMENT;
  if (rows > 1 && (x_stride < 0 || y_stride < cols)) return TBE_ERR_INVALID_ARGUMENT;
  NormArgs a{};
  a.x = x;
  a.x_stride = x_stride;
  a.weight = weight;
  a.bias = bias;
  a.y = y;
  a.y_stride = y_stride;
  a.stats = reinterpret_cast<float2*>(stats);
  a.rows = rows;
  a.cols = cols;
  a.eps = static_cast<float>(eps);
  a.count = static_cast<float>(cols);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t err = dtype == TBE_F32   ? launch_forward<kF32>(a, s)
                         : dtype == TBE_F16 ? launch_forward<kF16>(a, s)
                                            : launch_forward<kBF16>(a, s);
  return err == hipSuccess ? TBE_OK : TBE_ERR_HIP;
}

tbe_status tbe_layer_norm_backward(const void* x, int64_t x_stride, const float* stats, const void* grad,
                                   int64_t grad_stride, const void* weight, void* dx, int64_t dx_stride,
                                   void* dweight, void* dbias, int64_t rows, int64_t cols, int32_t dtype,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  const tbe_status st = check_sizes(rows, cols, dtype);
  if (st != TBE_OK) return st;
  const size_t e = dtype_bytes(dtype);
  if ((rows > 0 && (!x || !stats || !grad)) || !aligned_to(x, e) || !aligned_to(stats, 8) ||
      !aligned_to(grad, e) || !aligned_to(weight, e) || !aligned_to(dx, e) || !aligned_to(dweight, e) ||
      !aligned_to(dbias, e))
    return TBE_ERR_INVALID_ARGUMENT;
  if (rows > 1 && (x_stride < 0 || grad_stride < 0 || (dx && dx_stride < cols)))
    return TBE_ERR_INVALID_ARGUMENT;
  NormArgs a{};
  if (dweight || dbias) {
    if (!workspace || !aligned_to(workspace, 256)) return TBE_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < parts_bytes(rows, cols, dtype)) return TBE_ERR_WORKSPACE_TOO_SMALL;
    a.parts = static_cast<float*>(workspace);
  } else if (!dx || rows == 0) {
    return TBE_OK;
  }
  a.x = x;
  a.x_stride = x_stride;
  a.stats_in = reinterpret_cast<const float2*>(stats);
  a.grad = grad;
  a.g_stride = grad_stride;
  a.weight = weight;
  a.dx = dx;
  a.dx_stride = dx_stride;
  a.dweight = dweight;
  a.dbias = dbias;
  a.rows = rows;
  a.cols = cols;
  a.blocks = rows > 0 ? backward_blocks(rows, cols, dtype) : 0;
  a.count = static_cast<float>(cols);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t err = dtype == TBE_F32   ? launch_backward<kF32>(a, s)
                         : dtype == TBE_F16 ? launch_backward<kF16>(a, s)
                                            : launch_backward<kBF16>(a, s);
  return err == hipSuccess ? TBE_OK : TBE_ERR_HIP;
}

}  // extern "C"
