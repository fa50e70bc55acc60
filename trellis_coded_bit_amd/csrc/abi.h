// The C-ABI layer's error reporting, shared by its source files: one thread-local text behind
// trellis_last_error().
#pragma once
#include <hip/hip_runtime_api.h>

namespace trellis {

// Sets the calling thread's error text and returns `status`.
__attribute__((format(printf, 2, 3))) int abi_fail(int status, const char *fmt, ...);
void abi_clear();
// TRELLIS_OK, or TRELLIS_EHIP with the HIP error's text.
int abi_hip_status(hipError_t e, const char *what);

}  // namespace trellis
