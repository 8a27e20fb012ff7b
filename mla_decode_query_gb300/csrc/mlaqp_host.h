// Host-side services of the library shared by its translation units: the
// thread's error message and the device check.
#pragma once

#include <cuda_runtime.h>

#include <string>

namespace mlaqp {

// Record `msg` as this thread's last error and return `status`.
int host_fail(int status, const std::string& msg);
int host_fail_cuda(const char* what, cudaError_t e);

// The device (< 0: current) if it is an sm_103 GPU, with its SM count, else
// an error status.  Launches nothing.
int host_device(int device, int* resolved, int* sm_count);

}  // namespace mlaqp
