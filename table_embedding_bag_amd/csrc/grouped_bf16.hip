// grouped_bf16.hip -- the grouped linear layer's kernels for bf16 rows.
#include <hip/hip_runtime.h>

#define TBE_GROUPED_KERNELS
#include "grouped.hpp"

namespace tbe {
hipError_t launch_grouped_bf16(const GroupedArgs& a, bool backward, hipStream_t s) {
  return launch_grouped<kBF16>(a, backward, s);
}
}  // namespace tbe
