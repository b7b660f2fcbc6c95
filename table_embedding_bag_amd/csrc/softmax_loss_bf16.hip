// softmax_loss_bf16.hip -- the softmax loss's kernels for bf16 rows.
#include <hip/hip_runtime.h>

#include "loss_launch.hpp"

namespace tbe {
hipError_t launch_loss_bf16(const LossArgs& a, bool backward, hipStream_t s) {
  return launch_loss<kBF16>(a, backward, s);
}
}  // namespace tbe
