// Per-element mathematics of the gated linear recurrence h_t = a_t h_{t-1} + u_t.
//   log a = g, or -exp(A_log) softplus(g + dt_bias);   u = s sigma(i) x,   s = sqrt(1 - a^2) or 1.
// Written so that nothing cancels: a and a - 1 come from one polynomial, 1 - a^2 is -(a - 1)(2 + (a - 1)), softplus is
// max(z, 0) + log1p(exp(-|z|)), and sigma' is formed from exp(-|z|).
#pragma once

#include <cuda_runtime.h>

namespace gdn {
namespace glr {

// a = exp(x) and e = exp(x) - 1.  x = k ln 2 + r, |r| <= ln 2 / 2, with ln 2 split in two parts (Cody and Waite); p =
// exp(r) - 1 by the series up to r^7 / 7! (the next term is below 2^-25 of p); a = 2^k + 2^k p, e = (2^k - 1) + 2^k p.
// Rounding a once matters: a memory of n tokens multiplies a one-sided error of a by n (a decay taken from expf was off
// by 4e-5 after 10^4 tokens).  Below 2^-125 the decay is 0.
struct Decay { float a, e; };
__device__ __forceinline__ Decay decay(float x) {
    const float c = x < -87.f ? -87.f : (x > 88.f ? 88.f : x);      // (keeps NaN)
    const float t = fmaf(c, 1.4426950408889634f, 12582912.f);       // k in the low bits of 1.5 * 2^23 + k
    const float k = t - 12582912.f;
    const float r = fmaf(k, 2.1219444e-4f, fmaf(k, -0.693359375f, c));
    float q = fmaf(r, 1.f / 5040.f, 1.f / 720.f);
    q = fmaf(q, r, 1.f / 120.f);
    q = fmaf(q, r, 1.f / 24.f);
    q = fmaf(q, r, 1.f / 6.f);
    q = fmaf(q, r, 0.5f);
    const float p = fmaf(r * r, q, r);
    const float sc = __int_as_float((__float_as_int(t) << 23) + 0x3f800000);
    Decay d;
    d.a = fmaf(sc, p, sc);
    d.e = fmaf(sc, p, sc - 1.f);
    if (x < -87.f) d = {0.f, -1.f};
    return d;
}

// exp(-|z|) carries both softplus and sigma
struct Tail { float z, q; };
__device__ __forceinline__ Tail tail(float z) { return {z, expf(-fabsf(z))}; }

// log1p(q) = 2 atanh(w), w = q / (2 + q) <= 1/3, by the odd series up to w^13 (the next term is below 2^-25 of it)
__device__ __forceinline__ float softplus(const Tail& t) {
    const float w = __fdividef(t.q, 2.f + t.q), v = w * w;
    float s = fmaf(v, 2.f / 13.f, 2.f / 11.f);
    s = fmaf(s, v, 2.f / 9.f);
    s = fmaf(s, v, 2.f / 7.f);
    s = fmaf(s, v, 2.f / 5.f);
    s = fmaf(s, v, 2.f / 3.f);
    return fmaxf(t.z, 0.f) + fmaf(w * v, s, 2.f * w);
}
__device__ __forceinline__ float sigmoid(const Tail& t) { return __fdividef(t.z < 0.f ? t.q : 1.f, 1.f + t.q); }
__device__ __forceinline__ float sigmoid_slope(const Tail& t) {
    const float r = __fdividef(1.f, 1.f + t.q);
    return t.q * r * r;
}

__device__ __forceinline__ float root(float x) {
    float y;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// the input factor sqrt(1 - a^2)
__device__ __forceinline__ float input_factor(const Decay& d) { return root(fmaxf(-d.e * (2.f + d.e), 0.f)); }

}  // namespace glr
}  // namespace gdn
