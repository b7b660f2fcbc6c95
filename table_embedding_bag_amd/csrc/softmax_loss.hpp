// softmax_loss.hpp -- what the softmax loss's interface (softmax_loss.hip) and its kernels
// (loss_kernels.hpp, loss_narrow.hpp; softmax_loss_f32/f16/bf16.hip each compile them for
// one type) share.
#pragma once

#include "layers.hpp"
#include "loss_plan.hpp"

namespace tbe {

// Words of row_info for 64 rows: three of each, rounded up to a wave's 16-byte loads.
constexpr int kInfoBlock = 256;

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
  void* x_rows;           // [rows][x_width]: x, zeros where a row has no target
  int64_t x_width;
  void* dlogits;          // [rows][backward.width]: of one piece
  float* dx_parts;        // [splits][rows][K]; narrow rows: null with one split
  float* dw_parts;        // [splits][piece or vocab][K], or null with one split
  uint32_t* row_info;     // of every 64 rows their bases, targets and gradients
  float* factor;          // what the logits' gradients are multiplied by, what undoes it times
                          // the scale; fp16: its exponent
  void* dx;               // or null
  void* dtable;           // or null
};

hipError_t launch_loss_f32(const LossArgs& a, bool backward, hipStream_t s);
hipError_t launch_loss_f16(const LossArgs& a, bool backward, hipStream_t s);
hipError_t launch_loss_bf16(const LossArgs& a, bool backward, hipStream_t s);

}  // namespace tbe
