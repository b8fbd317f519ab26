// api_common.hpp -- what the C ABI layers (api.hip, api_tokens.hip) share:
// the calling thread's error message, the kernel-time events' lifetime and
// the environment switches.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mp3d {

// Stores the message of the calling thread's most recent failure and returns `code`.
int fail(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));

// MP3D_OK, or MP3D_EHIP with a message that names `what`.
int hip_status(hipError_t e, const char *what);

// MP3D_LOG=1 (read once)
bool log_enabled();

// Disarms the kernel-time events when a C-ABI call returns, whether or not
// it launched anything.
struct TimingScope {
    ~TimingScope();
};

constexpr int64_t kInt32Max = 2147483647;

}  // namespace mp3d
