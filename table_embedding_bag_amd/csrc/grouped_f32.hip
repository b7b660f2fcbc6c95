// grouped_f32.hip -- the grouped linear layer's kernels for f32 rows.
#include <hip/hip_runtime.h>

#define TBE_GROUPED_KERNELS
#include "grouped.hpp"

namespace tbe {
hipError_t launch_grouped_f32(const GroupedArgs& a, bool backward, hipStream_t s) {
  return launch_grouped<kF32>(a, backward, s);
}
}  // namespace tbe
