// grouped.hip -- a linear layer for each group of consecutive rows,
//   y_n = W_g x_n + bias_g                 for the rows n of group g,
// and its gradients
//   dx_n = W_g^T dy_n,   dW_g = sum_n dy_n x_n^T,   dbias_g = sum_n dy_n.
// Groups are ragged row ranges known on the device only (CSR offsets); sums
// are fp32 and rounded once.
//
// Large products are bound by the matrix cores, and those by the card's power:
// 32768 rows in 16 groups, 4096 -> 4096 bf16, forward and backward, take 3.1 ms (1.06
// PFLOP/s, the matrix cores busy in 65% and 59% of the cycles at the 1.7 GHz that random
// values leave; a library's product of the same sizes in equal groups runs at 1.1 to
// 1.2).  16384 rows in 8 groups of very different sizes, 1024 -> 4096, take 505 us (0.82
// PFLOP/s): five rounds of large tiles where 4.4 would do, and tiles of 128, which read
// twice the LDS bytes for the same outputs.  With few rows the weights' reading counts: 64 rows over 64 groups, 512 ->
// 2048, 19 us (4.6 TB/s of the weights that have rows).  Small ones are a few
// latencies: 8191 x 250 -> 130 fp32, both directions, 49 us in three launches.
// Times here and beside the kernels are of passes among others unless they say "kernel".
#include <hip/hip_runtime.h>

#include <algorithm>

#include "grouped.hpp"

using namespace tbe;

namespace {

hipError_t launch(const GroupedArgs& a, int32_t dtype, bool backward, hipStream_t s) {
  return dtype == TBE_F32   ? launch_grouped_f32(a, backward, s)
         : dtype == TBE_F16 ? launch_grouped_f16(a, backward, s)
                            : launch_grouped_bf16(a, backward, s);
}

RowLayout layout_of(const void* p, int64_t stride, int64_t width, int32_t dtype) {
  return row_layout(reinterpret_cast<uintptr_t>(p), stride, width, dtype_bytes(dtype));
}

// Longest rows and strides: 256 of them lie within a buffer descriptor's reach.
constexpr int64_t kMaxFeatures = int64_t{1} << 20;

// The chunks' sums of the weights' and the bias's gradients.
size_t backward_bytes_of(int64_t rows, int64_t groups, int64_t K, int64_t M, int32_t dtype) {
  return static_cast<size_t>(plan_grad_w(rows, groups, K, M, dtype).slots) *
         static_cast<size_t>(M * K + M) * sizeof(float);
}

tbe_status check_sizes(int64_t rows, int64_t groups, int64_t K, int64_t M, int32_t dtype) {
  if (rows < 0 || groups < 0 || K < 1 || M < 1 || !known_dtype(dtype))
    return TBE_ERR_INVALID_ARGUMENT;
  if (groups == 0 && rows > 0) return TBE_ERR_INVALID_ARGUMENT;
  // 31-bit rows, and grids of at most 2^31 threads whatever the tiles
  if (rows >= (int64_t{1} << 30) || groups > 65535 || K > kMaxFeatures || M > kMaxFeatures)
    return TBE_ERR_UNSUPPORTED;
  const int64_t tk = (K + 127) / 128, tm = (M + 127) / 128;
  if ((rows / 32 + groups) * std::max(tk, tm) > (int64_t{1} << 22) ||
      groups * tk * tm > (int64_t{1} << 22))
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
  *backward_bytes = backward_bytes_of(rows, groups, in_features, out_features, dtype);
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
  if (rows == 1) x_stride = in_features;  // a single row's stride says nothing
  if (x_stride > kMaxFeatures) return TBE_ERR_UNSUPPORTED;
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
  a.index64 = index_dtype == TBE_I64;
  a.layout = std::min(layout_of(x, x_stride, in_features, dtype),
                      layout_of(weight, in_features, in_features, dtype));
  return launch(a, dtype, false, static_cast<hipStream_t>(stream)) == hipSuccess
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
  if (rows <= 1) x_stride = in_features, grad_stride = out_features;
  if (x_stride > kMaxFeatures || grad_stride > kMaxFeatures) return TBE_ERR_UNSUPPORTED;
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
  if (dweight) {
    const GradWPlan plan = plan_grad_w(rows, groups, in_features, out_features, dtype);
    const size_t need = backward_bytes_of(rows, groups, in_features, out_features, dtype);
    if (need > 0 && (!workspace || !aligned_to(workspace, 256))) return TBE_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < need) return TBE_ERR_WORKSPACE_TOO_SMALL;
    a.chunk = plan.chunk;
    a.slots = plan.slots;
    a.parts = static_cast<float*>(workspace);
    a.bias_parts = a.parts + plan.slots * out_features * in_features;
  }
  a.index64 = index_dtype == TBE_I64;
  a.layout = std::min({layout_of(x, x_stride, in_features, dtype),
                       layout_of(weight, in_features, in_features, dtype),
                       layout_of(grad, grad_stride, out_features, dtype)});
  return launch(a, dtype, true, static_cast<hipStream_t>(stream)) == hipSuccess
             ? TBE_OK
             : TBE_ERR_HIP;
}

}  // extern "C"
