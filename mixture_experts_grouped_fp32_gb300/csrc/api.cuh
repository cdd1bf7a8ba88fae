// api.cuh — what the files with extern "C" entry points share (defined in moe_api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

// Records the calling thread's error message and returns `code`.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears the message and returns MOE_OK.
int ok();
// The current device must be compute capability 10.3; fills its SM count.
int check_device(int* num_sms);
// Failure-detection test hook: 1 with MOE_INJECT_STALL=1 in the environment.
int inject_stall();
// A launch's error as a return code.
int launched(cudaError_t e, const char* what);

inline bool aligned_to(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

}  // namespace moe
