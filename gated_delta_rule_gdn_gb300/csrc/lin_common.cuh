// Device pieces shared by the kernels of linear attention with a decay for each head: sequences, and the decays of a chunk.
#pragma once

#include "lin.h"
#include "mixer_common.cuh"

namespace gdn {
namespace lin {

// At the end of a kernel that was launched before the one before it had completed: the grid does not complete before that one, so
// that what waits for this kernel waits for both.  One block holds it; the others leave their SMs.
__device__ __forceinline__ void last_behind() {
    if (blockIdx.x == 0) mix::wait_behind();
}

// First token row and length of sequence n; malformed offsets are clamped into the tokens.
__device__ __forceinline__ void sequence(const int32_t* cu, int T, int n, int64_t& first, int& len) {
    if (cu) {
        const int a = mix::clamp_off(cu[n], T), b = mix::clamp_off(cu[n + 1], T);
        first = a;
        len = max(b - a, 0);
    } else {
        first = (int64_t)n * T;
        len = T;
    }
}

// The sequence that a slot of spans or segments of `size` tokens is one of (those of sequence n begin at first / size + n): the
// last that begins at or before it.
__device__ __forceinline__ int slot_sequence(const int32_t* cu, int N, int T, int size, int64_t slot) {
    int n = 0, top = (int)min(slot, (int64_t)N - 1), len;
    int64_t first;
    while (n < top) {
        const int mid = (n + top + 1) >> 1;
        sequence(cu, T, mid, first, len);
        if (first / size + mid <= slot) n = mid; else top = mid - 1;
    }
    return n;
}

// Rank in the launch -> sequence: packed sequences longest first, so that the longest walks do not start last (all lanes of a
// warp call it; up to 32 sequences, as many as the lanes).
__device__ __forceinline__ int by_length(const int32_t* cu, int n_seqs, int T, int rank) {
    if (!cu || n_seqs > 32) return rank;
    const int lane = threadIdx.x & 31;
    int at = -1;
    if (lane < n_seqs) {
        int64_t f;
        int mine, other;
        sequence(cu, T, lane, f, mine);
        at = 0;
        for (int m = 0; m < n_seqs; ++m) {
            sequence(cu, T, m, f, other);
            at += (other > mine) || (other == mine && m < lane);
        }
    }
    const unsigned hit = __ballot_sync(0xffffffffu, at == rank);
    return hit ? __ffs(hit) - 1 : rank;
}

// Log decays and their prefix sums are sums of two floats, hi + lo, so that differences within a chunk are exact to far below
// fp32's roundoff (a single float would be off by 2^-24 of the chunk's whole decay, so by 1e-5 and more next to strong decays;
// 64-bit arithmetic has a sixty-fourth of the rate here: a chunk's 128 prefix sums took longer than its products).
struct Log2 { float hi, lo; };
__device__ __forceinline__ Log2 add(Log2 a, Log2 b) {     // the sum's rounding error, then both joined anew
    const float s = __fadd_rn(a.hi, b.hi), t = __fsub_rn(s, a.hi);
    const float e = __fadd_rn(__fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(b.hi, t)), __fadd_rn(a.lo, b.lo));
    const float hi = __fadd_rn(s, e);
    return {hi, __fsub_rn(e, __fsub_rn(hi, s))};
}
__device__ __forceinline__ float minus(Log2 a, Log2 b) { return (a.hi - b.hi) + (a.lo - b.lo); }
// A log decay in base 2.  Below -1000 (2^-1000 is 0 in fp32 many times over) and at -inf it is -1000: sums of them stay finite,
// so that differences within a chunk do too.  A NaN stays one.
__device__ __forceinline__ Log2 log2_decay(float g) {
    constexpr float L = 1.44269502162933349609f, M = 1.92596299112661746888e-8f;     // log2(e) rounded, and the rest
    const float x = __fmul_rn(g, L);
    return x < -1000.f ? Log2{-1000.f, 0.f} : Log2{x, fmaf(g, L, -x) + __fmul_rn(g, M)};
}
// 2^x of a chunk's whole decay as the sum of two floats (below a half the second is 0), so that what a rounded factor is off by
// does not grow with the chunks of a long memory: 65,536 tokens with a decay of 1e-5 each would be off by 1e-5 and more.
struct Keep { float hi, lo; };
__device__ __forceinline__ Keep keep_of(Log2 x) {
    const float y = x.hi + x.lo, whole = exp2f(y);
    if (!(whole >= 0.5f)) return {whole, 0.f};
    const float rest = expm1f(0.69314718055994531f * y), hi = __fadd_rn(1.f, rest);
    return {hi, __fsub_rn(rest, __fsub_rn(hi, 1.f))};
}
__device__ __forceinline__ float keep(const Keep& k, float s, float add) { return fmaf(k.hi, s, fmaf(k.lo, s, add)); }
// Sums over the lanes up to this one.
__device__ __forceinline__ Log2 prefix(Log2 a, int lane) {
    for (int m = 1; m < 32; m <<= 1) {
        const Log2 b{__shfl_up_sync(0xffffffffu, a.hi, m), __shfl_up_sync(0xffffffffu, a.lo, m)};
        if (lane >= m) a = add(a, b);
    }
    return a;
}

}  // namespace lin
}  // namespace gdn
