// grouped.hip -- a linear layer for each group of consecutive rows,
//   y_n = W_g x_n + bias_g                 for the rows n of group g,
// and its gradients
//   dx_n = W_g^T dy_n,   dW_g = sum_n dy_n x_n^T,   dbias_g = sum_n dy_n.
// Groups are ragged row ranges known on the device only (CSR offsets); sums
// are fp32 and rounded once.
#include <hip/hip_runtime.h>

#include "layers.hpp"

using namespace tbe;

namespace {

constexpr int kTile = 64, kDepth = 16;

struct GroupedArgs {
  int64_t rows, groups, K, M;  // K = in_features, M = out_features
  const void* x;
  const void* weight;  // [groups, M, K]
  const void* bias;    // [groups, M] or null
  const void* offsets;
  void* y;
  const void* grad;    // [rows, M]
  void* dx;
  void* dw;
  void* db;
  int64_t x_stride, y_stride, grad_stride, dx_stride;
};

template <typename IT>
__device__ __forceinline__ int64_t offset_at(const GroupedArgs& a, int64_t g) {
  const int64_t o = static_cast<const IT*>(a.offsets)[g];
  return o < 0 ? 0 : (o > a.rows ? a.rows : o);
}

// The group and first row of row tile `tile` of all groups' tiles; false where
// there are fewer tiles.
template <typename IT>
__device__ bool find_tile(const GroupedArgs& a, int64_t tile, int64_t* group, int64_t* first,
                          int64_t* end) {
  int64_t lo = offset_at<IT>(a, 0);
  for (int64_t g = 0; g < a.groups; ++g) {
    const int64_t hi = offset_at<IT>(a, g + 1);
    const int64_t tiles = hi > lo ? (hi - lo + kTile - 1) / kTile : 0;
    if (tile < tiles) {
      *group = g;
      *first = lo + tile * kTile;
      *end = hi;
      return true;
    }
    tile -= tiles;
    lo = hi;
  }
  return false;
}

enum Product { kForward, kGradX, kGradW };

// One 64 x 64 tile of the output, 16 of the summed index at a time through LDS,
// 4 x 4 outputs a thread.
//   kForward  out[n, m] = sum_k x[n, k] W[g, m, k]
//   kGradX    out[n, k] = sum_m dy[n, m] W[g, m, k]
//   kGradW    out[m, k] = sum_n dy[n, m] x[n, k]
template <int ST, Product P, typename IT>
__global__ __launch_bounds__(kBlock) void grouped_tile(GroupedArgs a) {
  __shared__ float as[kDepth][kTile + 1], bs[kDepth][kTile + 1];
  int64_t g, first, end;
  if constexpr (P == kGradW) {
    g = blockIdx.z;
    first = offset_at<IT>(a, g);
    end = offset_at<IT>(a, g + 1);
    if (end < first) end = first;
  } else {
    if (!find_tile<IT>(a, blockIdx.y, &g, &first, &end)) return;
  }
  const int64_t i0 = P == kGradW ? static_cast<int64_t>(blockIdx.y) * kTile : first;
  const int64_t j0 = static_cast<int64_t>(blockIdx.x) * kTile;
  const int64_t rows = P == kGradW ? a.M : end;          // bounds of i, j and the summed index
  const int64_t cols = P == kForward ? a.M : a.K;
  const int64_t d0 = P == kGradW ? first : 0;
  const int64_t depth = P == kForward ? a.K : P == kGradX ? a.M : end;
  const char* wg = static_cast<const char*>(a.weight) + g * a.M * a.K * StorageTraits<ST>::bytes;
  const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
  float acc[4][4] = {};
  for (int64_t d = d0; d < depth; d += kDepth) {
    for (int e = threadIdx.x; e < kTile * kDepth; e += kBlock) {
      // neighbouring lanes read neighbouring elements of each operand's rows
      const int ad = P == kGradW ? e / kTile : e % kDepth, ai = P == kGradW ? e % kTile : e / kDepth;
      const int bd = P == kForward ? e % kDepth : e / kTile, bj = P == kForward ? e / kDepth : e % kTile;
      float av = 0.0f, bv = 0.0f;
      if (i0 + ai < rows && d + ad < depth)
        av = P == kForward  ? load_one<ST>(a.x, (i0 + ai) * a.x_stride + d + ad)
             : P == kGradX  ? load_one<ST>(a.grad, (i0 + ai) * a.grad_stride + d + ad)
                            : load_one<ST>(a.grad, (d + ad) * a.grad_stride + i0 + ai);
      if (j0 + bj < cols && d + bd < depth)
        bv = P == kForward  ? load_one<ST>(wg, (j0 + bj) * a.K + d + bd)
             : P == kGradX  ? load_one<ST>(wg, (d + bd) * a.K + j0 + bj)
                            : load_one<ST>(a.x, (d + bd) * a.x_stride + j0 + bj);
      as[ad][ai] = av;
      bs[bd][bj] = bv;
    }
    __syncthreads();
    for (int k = 0; k < kDepth; ++k) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += as[k][ti * 4 + i] * bs[k][tj + 16 * j];
    }
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t r = i0 + ti * 4 + i, c = j0 + tj + 16 * j;
      if (r >= rows || c >= cols) continue;
      float v = acc[i][j];
      if constexpr (P == kForward) {
        if (a.bias) v += load_one<ST>(a.bias, g * a.M + c);
        store_one<ST>(a.y, r * a.y_stride + c, v);
      } else if constexpr (P == kGradX) {
        store_one<ST>(a.dx, r * a.dx_stride + c, v);
      } else {
        store_one<ST>(a.dw, (g * a.M + r) * a.K + c, v);
      }
    }
}

// dbias: a workgroup sums 64 columns of one group, four rows at a time.
template <int ST, typename IT>
__global__ __launch_bounds__(kBlock) void grouped_bias_grad(GroupedArgs a) {
  __shared__ float part[4][64];
  const int64_t g = blockIdx.y;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + (threadIdx.x & 63);
  const int w = threadIdx.x >> 6;
  float sum = 0.0f;
  if (c < a.M)
    for (int64_t n = offset_at<IT>(a, g) + w; n < offset_at<IT>(a, g + 1); n += 4)
      sum += load_one<ST>(a.grad, n * a.grad_stride + c);
  part[w][threadIdx.x & 63] = sum;
  __syncthreads();
  if (w == 0 && c < a.M)
    store_one<ST>(a.db, g * a.M + c,
                  (part[0][threadIdx.x] + part[1][threadIdx.x]) +
                      (part[2][threadIdx.x] + part[3][threadIdx.x]));
}

unsigned tiles_of(int64_t n) { return static_cast<unsigned>((n + kTile - 1) / kTile); }

template <int ST, typename IT>
hipError_t launch_forward(const GroupedArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((grouped_tile<ST, kForward, IT>),
                     dim3(tiles_of(a.M), static_cast<unsigned>(a.rows / kTile + a.groups)),
                     dim3(kBlock), 0, s, a);
  return hipGetLastError();
}

template <int ST, typename IT>
hipError_t launch_backward(const GroupedArgs& a, hipStream_t s) {
  if (a.dx && a.rows > 0)
    hipLaunchKernelGGL((grouped_tile<ST, kGradX, IT>),
                       dim3(tiles_of(a.K), static_cast<unsigned>(a.rows / kTile + a.groups)),
                       dim3(kBlock), 0, s, a);
  if (a.dw)
    hipLaunchKernelGGL((grouped_tile<ST, kGradW, IT>),
                       dim3(tiles_of(a.K), tiles_of(a.M), static_cast<unsigned>(a.groups)),
                       dim3(kBlock), 0, s, a);
  if (a.db)
    hipLaunchKernelGGL((grouped_bias_grad<ST, IT>),
                       dim3(tiles_of(a.M), static_cast<unsigned>(a.groups)), dim3(kBlock), 0, s, a);
  return hipGetLastError();
}

template <int ST>
hipError_t launch(const GroupedArgs& a, int32_t index, bool back, hipStream_t s) {
  if (index == TBE_I64)
    return back ? launch_backward<ST, int64_t>(a, s) : launch_forward<ST, int64_t>(a, s);
  return back ? launch_backward<ST, int32_t>(a, s) : launch_forward<ST, int32_t>(a, s);
}

hipError_t launch(const GroupedArgs& a, int32_t dtype, int32_t index, bool back, hipStream_t s) {
  return dtype == TBE_F32   ? launch<kF32>(a, index, back, s)
         : dtype == TBE_F16 ? launch<kF16>(a, index, back, s)
                            : launch<kBF16>(a, index, back, s);
}

tbe_status check_sizes(int64_t rows, int64_t groups, int64_t K, int64_t M, int32_t dtype) {
  if (rows < 0 || groups < 0 || K < 1 || M < 1 || !known_dtype(dtype))
    return TBE_ERR_INVALID_ARGUMENT;
  if (groups == 0 && rows > 0) return TBE_ERR_INVALID_ARGUMENT;
  // grid dimensions of the launches below
  if (rows >= (int64_t{1} << 30) || groups > 65535 || K >= (int64_t{1} << 20) ||
      M >= (int64_t{1} << 20) || rows / kTile + groups > 65535)
    return TBE_ERR_UNSUPPORTED;
  return TBE_OK;
}

}  // namespace

extern "C" {

tbe_status tbe_grouped_linear_sizes(int64_t rows, int64_t groups, int64_t in_features,
                                    int64_t out_features, int32_t dtype, size_t* forward_bytes,
                                    size_t* backward_bytes) {
  if (!forward_bytes || !backward_bytes) return TBE_ERR_INVALID_ARGUMENT;
  const tbe_status st = check_sizes(rows, groups, in_features, out_features, dtype);
  if (st != TBE_OK) return st;
  *forward_bytes = 0;
  *backward_bytes = 0;
  return TBE_OK;
}

tbe_status tbe_grouped_linear(const void* x, int64_t x_stride, const void* weight, const void* bias,
                              const void* offsets, int32_t index_dtype, void* y, int64_t y_stride,
                              int64_t rows, int64_t groups, int64_t in_features,
                              int64_t out_features, int32_t dtype, void* workspace,
                              size_t workspace_bytes, void* stream) {
  const tbe_status st = check_sizes(rows, groups, in_features, out_features, dtype);
  if (st != TBE_OK) return st;
  if (index_dtype != TBE_I32 && index_dtype != TBE_I64) return TBE_ERR_INVALID_ARGUMENT;
  if (rows == 0) return TBE_OK;
  const size_t e = dtype_bytes(dtype);
  if (!x || !weight || !offsets || !y || !aligned_to(x, e) || !aligned_to(weight, e) ||
      !aligned_to(bias, e) || !aligned_to(y, e) ||
      !aligned_to(offsets, index_dtype == TBE_I64 ? 8 : 4))
    return TBE_ERR_INVALID_ARGUMENT;
  if (x_stride < 0 || (rows > 1 && y_stride < out_features)) return TBE_ERR_INVALID_ARGUMENT;
  GroupedArgs a{};
  a.rows = rows;
  a.groups = groups;
  a.K = in_features;
  a.M = out_features;
  a.x = x;
  a.x_stride = x_stride;
  a.weight = weight;
  a.bias = bias;
  a.offsets = offsets;
  a.y = y;
  a.y_stride = y_stride;
  return launch(a, dtype, index_dtype, false, static_cast<hipStream_t>(stream)) == hipSuccess
             ? TBE_OK
             : TBE_ERR_HIP;
}

tbe_status tbe_grouped_linear_backward(const void* x, int64_t x_stride, const void* weight,
                                       const void* offsets, int32_t index_dtype, const void* grad,
                                       int64_t grad_stride, void* dx, int64_t dx_stride,
                                       void* dweight, void* dbias, int64_t rows, int64_t groups,
                                       int64_t in_features, int64_t out_features, int32_t dtype,
                                       void* workspace, size_t workspace_bytes, void* stream) {
  const tbe_status st = check_sizes(rows, groups, in_features, out_features, dtype);
  if (st != TBE_OK) return st;
  if (index_dtype != TBE_I32 && index_dtype != TBE_I64) return TBE_ERR_INVALID_ARGUMENT;
  if (groups == 0) return TBE_OK;
  const size_t e = dtype_bytes(dtype);
  if (!offsets || !aligned_to(offsets, index_dtype == TBE_I64 ? 8 : 4) || !aligned_to(x, e) ||
      !aligned_to(weight, e) || !aligned_to(grad, e) || !aligned_to(dx, e) ||
      !aligned_to(dweight, e) || !aligned_to(dbias, e))
    return TBE_ERR_INVALID_ARGUMENT;
  if (rows > 0 && (!grad || (dx && !weight) || (dweight && !x))) return TBE_ERR_INVALID_ARGUMENT;
  if (x_stride < 0 || grad_stride < 0 || (dx && rows > 1 && dx_stride < in_features))
    return TBE_ERR_INVALID_ARGUMENT;
  GroupedArgs a{};
  a.rows = rows;
  a.groups = groups;
  a.K = in_features;
  a.M = out_features;
  a.x = x;
  a.x_stride = x_stride;
  a.weight = weight;
  a.offsets = offsets;
  a.grad = grad;
  a.grad_stride = grad_stride;
  a.dx = dx;
  a.dx_stride = dx_stride;
  a.dw = dweight;
  a.db = dbias;
  return launch(a, dtype, index_dtype, true, static_cast<hipStream_t>(stream)) == hipSuccess
             ? TBE_OK
             : TBE_ERR_HIP;
}

}  // extern "C"
