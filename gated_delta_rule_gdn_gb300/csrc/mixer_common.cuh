// Device helpers shared by the operators around the delta rule: element access in fp32 and packed-sequence lookup.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace gdn {
namespace mix {

using bf16 = __nv_bfloat16;

// A kernel launched behind another of the same call: its blocks may start once all of the first's have come to let_next(),
// and touch memory only after wait_behind(), which waits for the first to end with its writes visible.  (Sums of parameter
// gradients, forward and backward, against ordinary launches: convolution of 1000 tokens x 4096 channels 22.7 us and 25.1,
// recurrence 1000 x 2048 41.7 and 43.5, B4 T4096 D2048 277 and 280, norm of 16,384 tokens x 40 heads 172.7 and 174.0.)
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_behind() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// (`behind` false: an ordinary launch)
template <typename... P, typename... Q>
cudaError_t launch_behind(void (*kernel)(P...), dim3 blocks, int threads, size_t smem, bool behind, cudaStream_t s, Q... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = blocks;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = behind ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

__device__ __forceinline__ float ld(const float* p) { return *p; }
__device__ __forceinline__ float ld(const bf16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st(float* p, float x) { *p = x; }
__device__ __forceinline__ void st(bf16* p, float x) { *p = __float2bfloat16_rn(x); }

// N consecutive elements as one access (aligned to their size), kept in their storage type until they are used.
template <int BYTES> struct Raw;
template <> struct Raw<2> { using type = unsigned short; };
template <> struct Raw<4> { using type = unsigned int; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<16> { using type = uint4; };
template <typename T, int N>
struct Vec {
    using R = typename Raw<sizeof(T) * N>::type;
    union {
        R raw;
        T e[N];
    };
    __device__ __forceinline__ Vec() {}
    __device__ __forceinline__ void load(const T* p) { raw = *reinterpret_cast<const R*>(p); }
    __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<R*>(p) = raw; }
    __device__ __forceinline__ void zero() { raw = R{}; }
    __device__ __forceinline__ float get(int i) const;
    __device__ __forceinline__ void set(int i, float x);
};
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void of_f32(float* d, float x) { *d = x; }
__device__ __forceinline__ void of_f32(bf16* d, float x) { *d = __float2bfloat16_rn(x); }
template <typename T, int N> __device__ __forceinline__ float Vec<T, N>::get(int i) const { return to_f32(e[i]); }
template <typename T, int N> __device__ __forceinline__ void Vec<T, N>::set(int i, float x) { of_f32(&e[i], x); }

// d = a * b + c (and d = a * b) over N floats, two to an instruction where N is even.
template <int N>
__device__ __forceinline__ void fma_row(float (&d)[N], const float (&a)[N], const float (&b)[N], const float (&c)[N]) {
    if constexpr (N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 2)
            asm("{\n\t.reg .b64 x, y, z;\n\t"
                "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
                "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
                : "=f"(d[i]), "=f"(d[i + 1])
                : "f"(a[i]), "f"(a[i + 1]), "f"(b[i]), "f"(b[i + 1]), "f"(c[i]), "f"(c[i + 1]));
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) d[i] = fmaf(a[i], b[i], c[i]);
    }
}
template <int N>
__device__ __forceinline__ void mul_row(float (&d)[N], const float (&a)[N], const float (&b)[N]) {
    if constexpr (N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 2)
            asm("{\n\t.reg .b64 x, y;\n\t"
                "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
                "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
                : "=f"(d[i]), "=f"(d[i + 1])
                : "f"(a[i]), "f"(a[i + 1]), "f"(b[i]), "f"(b[i + 1]));
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) d[i] = a[i] * b[i];
    }
}

template <int N>
__device__ __forceinline__ void add_row(float (&d)[N], const float (&a)[N], const float (&b)[N]) {
    if constexpr (N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 2)
            asm("{\n\t.reg .b64 x, y;\n\t"
                "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
                "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
                : "=f"(d[i]), "=f"(d[i + 1])
                : "f"(a[i]), "f"(a[i + 1]), "f"(b[i]), "f"(b[i + 1]));
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) d[i] = a[i] + b[i];
    }
}

// Copy V elements into shared memory without waiting (or zeros); the copying thread alone reads them.
template <typename T, int V>
__device__ __forceinline__ void copy_async(Vec<T, V>* dst, const T* src, bool in) {
    constexpr int N = sizeof(T) * V;
    if constexpr (N >= 4) {
        const unsigned d = static_cast<unsigned>(__cvta_generic_to_shared(dst));
        const int size = in ? N : 0;
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(d), "l"(src), "n"(N), "r"(size) : "memory");
    } else {                                     // (two bytes: no asynchronous form)
        if (in) dst->load(src); else dst->zero();
    }
}
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// wait until at most N of the closed groups are under way
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Packed sequences: the one that token t belongs to, with its first token and one past its last.  Every offset is
// clamped into [0, T], and the answer always satisfies 0 <= first <= t < end <= T, so a malformed array cannot lead
// an access outside the tensors.
struct Span { int n, first, end; };
__device__ __forceinline__ int clamp_off(int v, int T) { return min(max(v, 0), T); }
__device__ __forceinline__ Span span_of(const int32_t* cu, int n_seqs, int T, int t) {
    int lo = 0, hi = n_seqs - 1;                  // the largest n with cu[n] <= t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (clamp_off(cu[mid], T) <= t) lo = mid; else hi = mid - 1;
    }
    Span s;
    s.n = lo;
    s.first = min(clamp_off(cu[lo], T), t);
    s.end = max(clamp_off(cu[lo + 1], T), t + 1);
    return s;
}

}  // namespace mix
}  // namespace gdn
