// Status helpers of the C ABI's translation units (host only).
#pragma once

#include "../../include/kvq.h"

#include <cuda_runtime.h>

namespace kvq {

// set the thread's last-error message and return st
kvq_status fail(kvq_status st, const char* fmt, ...);
kvq_status cuda_fail(cudaError_t e, const char* what);

}  // namespace kvq
