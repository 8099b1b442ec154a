// Helpers of the C-ABI layer, shared by its translation units: the
// thread-local error text, the device check and the launch status.  Defined in
// hq_api.cpp; nothing here is exported.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hq.h"
#include "hq_internal.hpp"

namespace hq {
namespace api {

constexpr int64_t kI32 = 2147483647LL;

// Sets this thread's error text and returns `code`; ok() clears it.
__attribute__((visibility("hidden"))) hq_status fail(hq_status code, const char* fmt, ...);
__attribute__((visibility("hidden"))) hq_status ok();
// The current device's properties; HQ_ERR_DEVICE when it is not gfx950.
__attribute__((visibility("hidden"))) hq_status current_device(DeviceInfo* out);
// HQ_OK or HQ_ERR_LAUNCH from the result of a launch.
__attribute__((visibility("hidden"))) hq_status launched(hipError_t e, const char* what);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace api
}  // namespace hq
