// softmax_loss.hip -- the softmax cross entropy of rows x [N, K] against a table W [V, K]
// of which each row has a target:
//   z = scale x W^T,   lse_n = ln sum_v exp(z_nv),   loss_n = lse_n - z_n,target,
// and its gradients, with d_nv = g_n (exp(z_nv - lse_n) - [v = target_n]),
//   dx = scale d W,   dW = scale d^T x.
// The logits z are never kept: the forward pass reduces each tile of them to a row's
// sum of powers, the backward pass computes them again, one piece of the vocabulary at a
// time, and holds that piece's d in the rows' type (the one rounding beside the outputs')
// for the two products that read it: the matrix cores take 2-byte operands ten times as fast as
// fp32 ones.  2048 rows, 100000 x 128, bf16: dx is off by 0.0024 of its norm, dtable by 0.0021, where
// the rounding of the output alone makes 0.0017 of both.
//
// The matrix cores bound it: four products of 2 N V K operations, five for narrow rows
// (loss_narrow.hpp), whose gradients each compute the logits.  16384 rows, 131072 outputs of 512,
// fp16: forward 2.2 ms (1.0 PFLOP/s), backward 7.2 ms: 8 pieces of 0.40 ms for the logits'
// gradients (0.68, with 512 MB to write), 0.26 for the table's (1.08), 0.29 for x's (0.95); pieces
// of 32 to 256 MB, which the last cache could hold, were slower.
#include <hip/hip_runtime.h>

#include <cmath>

#include "softmax_loss.hpp"

using namespace tbe;

namespace {

hipError_t launch(const LossArgs& a, int32_t dtype, bool backward, hipStream_t s) {
  return dtype == TBE_F32   ? launch_loss_f32(a, backward, s)
         : dtype == TBE_F16 ? launch_loss_f16(a, backward, s)
                            : launch_loss_bf16(a, backward, s);
}

// Longest rows and strides: 256 of them lie within a buffer descriptor's reach.
constexpr int64_t kMaxWidth = int64_t{1} << 20;

tbe_status check_sizes(int64_t rows, int64_t vocab, int64_t K, int32_t dtype) {
  if (rows < 0 || vocab < 1 || K < 1 || !known_dtype(dtype)) return TBE_ERR_INVALID_ARGUMENT;
  // grids of at most 2^31 threads whatever the tiles
  if (rows > (int64_t{1} << 24) || vocab > (int64_t{1} << 30) || K > kMaxWidth ||
      rows > (int64_t{1} << 33) / K || vocab > (int64_t{1} << 36) / K)
    return TBE_ERR_UNSUPPORTED;
  return TBE_OK;
}

// Carves a workspace; with a null base it only counts.
struct Carver {
  char* base;
  size_t used = 0;
  void* take(int64_t bytes) {
    void* p = base ? base + used : nullptr;
    used += (static_cast<size_t>(bytes) + 255) / 256 * 256;
    return p;
  }
};

void carve_forward(LossArgs* a, Carver* c) {
  a->parts = static_cast<float2*>(c->take(a->forward.segments * a->rows * 8));
  a->target_logit = static_cast<float*>(c->take(a->rows * 4));
}

void carve_backward(LossArgs* a, int32_t dtype, bool dx, bool dtable, Carver* c) {
  const LossBackwardPlan& p = a->backward;
  const int64_t bytes = dtype_bytes(dtype);
  a->factor = static_cast<float*>(c->take(12));
  a->x_width = padded_width(a->K, bytes);
  a->x_rows = c->take(a->rows * a->x_width * bytes);
  a->row_info = static_cast<uint32_t*>(c->take(ceil_div(a->rows, 64) * kInfoBlock * 4));
  if (p.narrow) {
    if (dx && p.nx.splits > 1)
      a->dx_parts = static_cast<float*>(c->take(p.nx.splits * a->rows * a->K * 4));
    if (dtable && p.nw.splits > 1)
      a->dw_parts = static_cast<float*>(c->take(p.nw.splits * a->vocab * a->K * 4));
    return;
  }
  a->dlogits = c->take(a->rows * p.width * bytes);
  a->dx_parts = dx ? static_cast<float*>(c->take(p.x.splits * a->rows * a->K * 4)) : nullptr;
  a->dw_parts =
      dtable && p.w.splits > 1 ? static_cast<float*>(c->take(p.w.splits * p.piece * a->K * 4)) : nullptr;
}

LossArgs args_of(int64_t rows, int64_t vocab, int64_t K, double scale) {
  LossArgs a{};
  a.rows = rows;
  a.vocab = vocab;
  a.K = K;
  a.scale = static_cast<float>(scale);
  a.exponent = static_cast<float>(scale * 1.44269504088896340736);
  return a;
}

bool takes_narrow(const LossArgs& a, int32_t dtype) {
  return narrow_rows(a.K, dtype) && a.table_layout == kChunkRows;
}

// What both calls check of their inputs, with which it completes the arguments.
tbe_status check_inputs(LossArgs* a, const void* x, int64_t x_stride, const void* table,
                        int64_t table_stride, const void* targets, int32_t index_dtype, int32_t dtype) {
  if (index_dtype != TBE_I32 && index_dtype != TBE_I64) return TBE_ERR_INVALID_ARGUMENT;
  if (!(a->scale > 0.0f) || !std::isfinite(a->exponent)) return TBE_ERR_INVALID_ARGUMENT;
  const size_t e = dtype_bytes(dtype);
  if (a->rows > 0 && (!x || !table || !targets)) return TBE_ERR_INVALID_ARGUMENT;
  if (!aligned_to(x, e) || !aligned_to(table, e) ||
      !aligned_to(targets, index_dtype == TBE_I64 ? 8 : 4) || x_stride < 0 || table_stride < 0)
    return TBE_ERR_INVALID_ARGUMENT;
  if (a->rows <= 1) x_stride = a->K;  // a single row's stride says nothing
  if (a->vocab == 1) table_stride = a->K;
  if (x_stride > kMaxWidth || table_stride > kMaxWidth) return TBE_ERR_UNSUPPORTED;
  a->x = x;
  a->x_stride = x_stride;
  a->table = table;
  a->table_stride = table_stride;
  a->targets = targets;
  a->index64 = index_dtype == TBE_I64;
  a->table_layout = row_layout(reinterpret_cast<uintptr_t>(table), table_stride, a->K, e);
  a->layout = std::min<int32_t>(a->table_layout,
                                row_layout(reinterpret_cast<uintptr_t>(x), x_stride, a->K, e));
  return TBE_OK;
}

}  // namespace

extern "C" {

tbe_status tbe_softmax_loss_sizes(int64_t rows, int64_t vocab, int64_t dim, int32_t dtype,
                                  size_t* forward_bytes, size_t* backward_bytes) {
  if (!forward_bytes || !backward_bytes) return TBE_ERR_INVALID_ARGUMENT;
  const tbe_status st = check_sizes(rows, vocab, dim, dtype);
  if (st != TBE_OK) return st;
  *forward_bytes = 0;
  *backward_bytes = 256;
  if (rows == 0) return TBE_OK;
  LossArgs a = args_of(rows, vocab, dim, 1.0);
  *backward_bytes = 0;
  for (int narrow = 0; narrow <= (narrow_rows(dim, dtype) ? 1 : 0); ++narrow) {  // by the alignment
    a.forward = plan_loss_forward(rows, vocab, dim, narrow, dtype);
    a.backward = plan_loss_backward(rows, vocab, dim, narrow, dtype);
    Carver f{nullptr}, b{nullptr};
    carve_forward(&a, &f);
    carve_backward(&a, dtype, true, true, &b);
    *forward_bytes = std::max(*forward_bytes, f.used);
    *backward_bytes = std::max(*backward_bytes, b.used);
  }
  return TBE_OK;
}

tbe_status tbe_softmax_loss(const void* x, int64_t x_stride, const void* table, int64_t table_stride,
                            const void* targets, int32_t index_dtype, double scale, float* loss,
                            float* lse, int64_t rows, int64_t vocab, int64_t dim, int32_t dtype,
                            void* workspace, size_t workspace_bytes, void* stream) {
  tbe_status st = check_sizes(rows, vocab, dim, dtype);
  if (st != TBE_OK) return st;
  LossArgs a = args_of(rows, vocab, dim, scale);
  st = check_inputs(&a, x, x_stride, table, table_stride, targets, index_dtype, dtype);
  if (st != TBE_OK || rows == 0) return st;
  if (!loss || !lse || !aligned_to(loss, 4) || !aligned_to(lse, 4)) return TBE_ERR_INVALID_ARGUMENT;
  a.loss = loss;
  a.lse = lse;
  a.forward = plan_loss_forward(rows, vocab, dim, takes_narrow(a, dtype), dtype);
  Carver c{static_cast<char*>(workspace)};
  carve_forward(&a, &c);
  if (!workspace || !aligned_to(workspace, 256)) return TBE_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < c.used) return TBE_ERR_WORKSPACE_TOO_SMALL;
  return launch(a, dtype, false, static_cast<hipStream_t>(stream)) == hipSuccess ? TBE_OK
                                                                                 : TBE_ERR_HIP;
}

tbe_status tbe_softmax_loss_backward(const void* x, int64_t x_stride, const void* table,
                                     int64_t table_stride, const void* targets, int32_t index_dtype,
                                     double scale, const float* lse, const float* grad, void* dx,
                                     void* dtable, int64_t rows, int64_t vocab, int64_t dim,
                                     int32_t dtype, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  tbe_status st = check_sizes(rows, vocab, dim, dtype);
  if (st != TBE_OK) return st;
  LossArgs a = args_of(rows, vocab, dim, scale);
  st = check_inputs(&a, x, x_stride, table, table_stride, targets, index_dtype, dtype);
  if (st != TBE_OK) return st;
  const size_t e = dtype_bytes(dtype);
  if ((rows > 0 && (!lse || !grad)) || !aligned_to(lse, 4) || !aligned_to(grad, 4) ||
      !aligned_to(dx, e) || !aligned_to(dtable, e))
    return TBE_ERR_INVALID_ARGUMENT;
  if (!dtable && (!dx || rows == 0)) return TBE_OK;
  a.lse_in = lse;
  a.grad = grad;
  a.dx = rows > 0 ? dx : nullptr;
  a.dtable = dtable;
  Carver c{static_cast<char*>(workspace)};
  if (rows > 0) {
    a.backward = plan_loss_backward(rows, vocab, dim, takes_narrow(a, dtype), dtype);
    carve_backward(&a, dtype, dx, dtable, &c);
  } else {
    a.factor = static_cast<float*>(c.take(12));
  }
  if (!workspace || !aligned_to(workspace, 256)) return TBE_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < c.used) return TBE_ERR_WORKSPACE_TOO_SMALL;
  return launch(a, dtype, true, static_cast<hipStream_t>(stream)) == hipSuccess ? TBE_OK
                                                                                : TBE_ERR_HIP;
}

}  // extern "C"
