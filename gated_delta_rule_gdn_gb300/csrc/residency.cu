// Host side of persistent kernels: resident blocks (residency.h).

#include "residency.h"

#include "internal.h"

namespace gdn {

cudaError_t Residency::get(const void* kernel, int threads, int smem, int* blocks) {
    int dev = 0, sms = 0, per = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < kDevices && (*blocks = known[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
    cudaFuncAttributes attr{};
    e = cudaFuncGetAttributes(&attr, kernel);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)(kMaxSmemPerBlock - attr.sharedSizeBytes));
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, smem);
    if (e != cudaSuccess) return e;
    *blocks = sms * (per > 0 ? per : 1);
    if (dev < kDevices) known[dev].store(*blocks, std::memory_order_relaxed);
    return cudaSuccess;
}

}  // namespace gdn
