// ops.cuh -- what the translation units of the serving operators share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <string>

namespace m3 {

// The thread-local message behind m3_last_error (m3.cu).
int set_error(int code, const std::string& msg);

// log2 of a page size the operators take (a power of two, 16..1024), or -1.
int page_shift(int page);

// SMs of the current device.
int sm_count();

}  // namespace m3
