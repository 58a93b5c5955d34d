// Host pieces shared by the C ABI sources: the status helpers behind
// fp8mm_last_error and the limits of pointers and leading dimensions.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8mm.h"

namespace fp8mm {
namespace api {

// Sets the calling thread's message and returns the status.
fp8mm_status fail(fp8mm_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears the message; FP8MM_OK.
fp8mm_status ok();
// A launch's result as a status: FP8MM_ERUNTIME with HIP's text on failure.
fp8mm_status from_hip(hipError_t e, const char* what);
const char* last_error();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int64_t kMaxLd = int64_t(1) << 22;

}  // namespace api
}  // namespace fp8mm
