// softmax_loss_f32.hip -- the softmax loss's kernels for fp32 rows.
#include <hip/hip_runtime.h>

#include "loss_launch.hpp"

namespace tbe {
hipError_t launch_loss_f32(const LossArgs& a, bool backward, hipStream_t s) {
  return launch_loss<kF32>(a, backward, s);
}
}  // namespace tbe
