// What the host-side files of the C ABI share.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/stce.h"

namespace stce {

// Records the message stce_last_error() returns on this thread; returns s.
stce_status fail(stce_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
stce_status hip_fail(hipError_t e, const char* what);

}  // namespace stce
