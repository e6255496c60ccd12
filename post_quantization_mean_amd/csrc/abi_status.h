// The thread-local error state behind awq_last_error(), shared by the files that implement the C ABI.
#pragma once

#include <hip/hip_runtime.h>

namespace awq {

// Records a formatted detail for the calling thread and returns `status`.
int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int ok();  // clears the detail, returns AWQ_OK
int hip_fail(hipError_t e, const char* where);

}  // namespace awq
