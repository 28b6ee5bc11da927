// How many blocks of a kernel the current device holds at once (persistent kernels launch no more).
#pragma once

#include <cuda_runtime_api.h>
#include <atomic>

namespace gdn {

struct Residency {
    static constexpr int kDevices = 64;          // devices whose answer is kept; others are asked every time
    std::atomic<int> known[kDevices]{};
    // With this many threads and bytes of dynamic shared memory a block; the kernel may use all that a block can have.
    // *blocks is 1 or more where this returns cudaSuccess, and a failed query returns its own error.
    cudaError_t get(const void* kernel, int threads, int smem, int* blocks);
};

}  // namespace gdn
