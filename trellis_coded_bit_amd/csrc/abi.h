// What the C-ABI layer's source files share: error reporting (one thread-local text behind
// trellis_last_error()) and the turns of host threads at a workspace.
#pragma once
#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <mutex>

namespace trellis {

// Sets the calling thread's error text and returns `status`.
__attribute__((format(printf, 2, 3))) int abi_fail(int status, const char *fmt, ...);
void abi_clear();
// TRELLIS_OK, or TRELLIS_EHIP with the HIP error's text.
int abi_hip_status(hipError_t e, const char *what);

// Held while a call that uses a workspace's scratch enqueues its launches.  A stream keeps the order
// in which launches reach it, so what one launch leaves in the scratch for the call's next is still
// there only if no other thread's call reaches the stream in between.  Workspaces share 64 locks by
// address: two that meet in one wait for a few launches, no more.
class WorkspaceTurn {
 public:
  explicit WorkspaceTurn(const void *ws) : lock_(lock_of(ws)) {}

 private:
  static std::mutex &lock_of(const void *ws) {
    static std::mutex locks[64];
    return locks[(reinterpret_cast<uintptr_t>(ws) >> 8) * 0x9E3779B97F4A7C15ull >> 58];
  }
  std::lock_guard<std::mutex> lock_;
};

}  // namespace trellis
