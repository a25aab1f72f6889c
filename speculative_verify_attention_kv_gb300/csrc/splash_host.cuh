// Host helpers shared by the C ABI's translation units.
#pragma once

#include <cuda_runtime.h>

namespace splash {

// SM count of the current device (looked up once per device), 0 on failure.
int device_sm_count();

// Counts a successful launch (splash_launch_count) and passes the result on.
cudaError_t counted(cudaError_t e);

// Limit of the tensor-core kernels' internal waits (splash_set_wait_limit_ns).
unsigned long long wait_limit_ns();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace splash
