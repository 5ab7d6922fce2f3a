// Host-side checks shared by the translation units of the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe_nvfp4.h"

namespace moe {

// Records the calling thread's error message and returns the status.
moe_status fail(moe_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// The current device must be gfx950; checked once per device id.
moe_status check_device();
// MOE_OK, or MOE_ERR_LAUNCH with the HIP error's message.
moe_status launched(hipError_t e, const char* what);

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

}  // namespace moe
