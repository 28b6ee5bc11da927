// Error reporting and argument checks shared by the C ABI's translation units (defined in api.cu).
#pragma once

#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "../../include/gdn.h"

namespace gdn {

// Record a message for gdn_last_error() and return the status.
gdn_status fail(gdn_status s, const char* fmt, ...);
gdn_status ok();
gdn_status cuda_fail(cudaError_t e, const char* what);

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool dtype_ok(gdn_dtype d) { return d == GDN_F32 || d == GDN_BF16; }

}  // namespace gdn
