// Host helpers of the C ABI shared by its sources (defined in api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <mutex>

#include "w8a16.h"

namespace w8a16 {

// Split-K workspace and arrival counters of one (device, stream).  The
// counters are zeroed once at allocation; every kernel that uses them
// leaves them at zero again.
struct Workspace {
    float *ws = nullptr;
    uint64_t ws_bytes = 0;
    uint32_t *counters = nullptr;
    uint32_t counter_count = 0;
};

// One call's use of a workspace.  The launches of a call hand each other
// partial results through it, and another thread's on the same stream must not
// come between them: held until the last of them is enqueued.
using WorkspaceHold = std::unique_lock<std::mutex>;

// Record a HIP failure of `what`; returns W8A16_ERR_HIP.
int hip_fail(hipError_t e, const char *what);
// W8A16_OK, or W8A16_ERR_ENV for a bad diagnostic setting.
int check_levers(const char *entry);
// Whether W8A16_LOG is on, and a line for it (printed once per process).
bool log_enabled();
void log_line(const char *line);
// Success epilogue of a call that enqueued work.
int launched(hipStream_t stream);
int device_cu_count(int dev, uint32_t *out);
// Workspace with at least the plan's workspace_bytes and counter_count.
int get_workspace(int dev, hipStream_t stream, const w8a16_plan_t &plan, Workspace *out, WorkspaceHold *hold);

// Status of the exception being handled: none (of an allocation in the maps and
// strings behind the helpers, of a mutex) leaves a C entry.
int caught(const char *entry) noexcept;
template <class F> int guarded(const char *entry, F f) noexcept
{
    try {
        return f();
    } catch (...) {
        return caught(entry);
    }
}

}  // namespace w8a16
