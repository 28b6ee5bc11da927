// Argument checks shared by the entry points of the operators around and beside the delta rule.
#pragma once

#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "../../include/gdn.h"
#include "api_util.h"

namespace {

using gdn::aligned;
using gdn::cuda_fail;
using gdn::dtype_ok;
using gdn::fail;
using gdn::ok;

inline size_t size_of(gdn_dtype d) { return d == GDN_BF16 ? 2 : 4; }

// Rows are counted in 32 bits and elements in 64.
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 65536;

// A tensor the call needs: present, and aligned to its element size.
inline gdn_status need(const char* fn, const char* name, const void* p, size_t es) {
    if (!p) return fail(GDN_ERR_INVALID_ARG, "%s: %s must be non-NULL", fn, name);
    if (!aligned(p, es)) return fail(GDN_ERR_INVALID_ARG, "%s: %s is not aligned to its element size", fn, name);
    return GDN_OK;
}
// One it may have.
inline gdn_status may(const char* fn, const char* name, const void* p, size_t es) {
    return p ? need(fn, name, p, es) : GDN_OK;
}

#define GDN_TRY(expr)                        \
    do {                                     \
        const gdn_status st_ = (expr);       \
        if (st_ != GDN_OK) return st_;       \
    } while (0)

// The caller's workspace, checked, or one allocated on the stream (freed by the destructor there).
struct Workspace {
    void* ptr = nullptr;
    bool own = false;
    cudaStream_t s = nullptr;
    gdn_status get(const char* fn, void* given, size_t given_bytes, size_t bytes, cudaStream_t stream) {
        s = stream;
        if (given) {
            if (given_bytes < bytes)
                return fail(GDN_ERR_INVALID_ARG, "%s: workspace of %zu bytes is smaller than the %zu needed", fn,
                            given_bytes, bytes);
            if (!aligned(given, 256)) return fail(GDN_ERR_INVALID_ARG, "%s: workspace is not 256-byte aligned", fn);
            ptr = given;
            return GDN_OK;
        }
        if (bytes == 0) return GDN_OK;
        const cudaError_t e = cudaMallocAsync(&ptr, bytes, s);
        if (e != cudaSuccess) {
            ptr = nullptr;
            return cuda_fail(e, fn);
        }
        own = true;
        return GDN_OK;
    }
    cudaError_t release() {
        const bool mine = own;
        own = false;
        return mine ? cudaFreeAsync(ptr, s) : cudaSuccess;
    }
    ~Workspace() { (void)release(); }
};

inline gdn_status finish(const char* fn, cudaError_t e, Workspace& ws) {
    const cudaError_t e2 = ws.release();
    if (e == cudaSuccess) e = e2;
    return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}

}  // namespace
