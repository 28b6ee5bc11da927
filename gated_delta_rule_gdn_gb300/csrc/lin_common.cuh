// Device pieces shared by the kernels of linear attention with a decay for each head: sequences, and the decays of a chunk.
#pragma once

#include "lin.h"
#include "mixer_common.cuh"

namespace gdn {
namespace lin {

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

// A log decay in base 2.  Below -1000 (2^-1000 is 0 in fp32 many times over) and at -inf it is -1000: sums of them stay finite,
// so that differences within a chunk do too.  A NaN stays one.
__device__ __forceinline__ double log2_decay(float g) {
    const double x = (double)g * 1.4426950408889634074;
    return x < -1000.0 ? -1000.0 : x;
}
// 2^x for x <= 0 given as a double (a difference of prefix sums, exact to far below fp32's roundoff; in fp32 the sums themselves
// would be off by 2^-24 of the chunk's whole decay, so by 1e-5 and more next to strong decays)
__device__ __forceinline__ float exp2_of(double x) { return exp2f((float)x); }

}  // namespace lin
}  // namespace gdn
