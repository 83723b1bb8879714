// Status helpers of the C ABI, shared by the files that define entry points.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/expert_ffn.h"

namespace moe {

// keeps "<fn>: <what>" for moe_last_error() on this thread and returns st
__attribute__((format(printf, 3, 4))) moe_status fail(moe_status st, const char* fn, const char* fmt, ...);
// MOE_OK, or MOE_E_HIP with the runtime's error string
moe_status hip_status(const char* fn, hipError_t e);

inline bool dt_ok(int32_t d) { return d == MOE_F32 || d == MOE_BF16; }
inline bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace moe
