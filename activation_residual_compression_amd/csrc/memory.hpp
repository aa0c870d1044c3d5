// Host side: device memory of the plans.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>

namespace rc {

// False, and null, where there is not as much. The runtime keeps the error of a failed call until it is asked for, and
// would report it at the caller's next launch, whoever's that is.
inline bool allocate(void** p, size_t bytes) {
  if (hipMalloc(p, bytes) == hipSuccess) return true;
  *p = nullptr;
  (void)hipGetLastError();
  return false;
}

}  // namespace rc
