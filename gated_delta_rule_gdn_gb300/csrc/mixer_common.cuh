// Device helpers shared by the operators around the delta rule: element access in fp32 and packed-sequence lookup.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace gdn {
namespace mix {

using bf16 = __nv_bfloat16;

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
