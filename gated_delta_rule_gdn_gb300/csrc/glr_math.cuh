// Per-element mathematics of the gated linear recurrence h_t = a_t h_{t-1} + u_t.
//   log a = g, or -exp(A_log) softplus(g + dt_bias);   u = s sigma(i) x,   s = sqrt(1 - a^2) or 1.
// Written so that nothing cancels: a and a - 1 come from one polynomial, 1 - a^2 is -(a - 1)(2 + (a - 1)), softplus is
// max(z, 0) + log1p(exp(-|z|)).  The scans spend about as long on these as on their memory traffic, so each is kept to
// as few instructions as its accuracy allows; the polynomials are minimax fits (Remez exchange) of this file's own;
// the bounds stated with them are of the fp32 coefficients as they stand here, before the rounding of the evaluation.
#pragma once

#include <cuda_runtime.h>

namespace gdn {
namespace glr {

constexpr float kLog2e = 1.4426950408889634f;

// Single-instruction approximations (relative error about 2^-22), flushing what is below 2^-126 to zero, and maxima that
// keep NaN.
__device__ __forceinline__ float ex2(float x) { float y; asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x)); return y; }
__device__ __forceinline__ float rcp(float x) { float y; asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x)); return y; }
__device__ __forceinline__ float rsq(float x) { float y; asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x)); return y; }
__device__ __forceinline__ float root(float x) { float y; asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x)); return y; }
__device__ __forceinline__ float max_nan(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float min_nan(float x, float y) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

// Two fp32 numbers to an instruction (the pair in one 64-bit register).
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack(float x, float y) { f2 r; asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y)); return r; }
__device__ __forceinline__ f2 both_of(float x) { return pack(x, x); }
__device__ __forceinline__ void unpack(f2 r, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(r)); }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) { f2 r; asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c)); return r; }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) { f2 r; asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b)); return r; }
__device__ __forceinline__ f2 add2(f2 a, f2 b) { f2 r; asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b)); return r; }

// a = exp(x) and e = exp(x) - 1 for x <= 88.  x = k ln 2 + r, |r| <= ln 2 / 2, with ln 2 split in two parts (Cody and
// Waite); p = exp(r) - 1 = r + r^2 Q(r), off by less than 2^-27.7; a = 2^k + 2^k p, e = (2^k - 1) + 2^k p.
// Rounding a once matters: a memory of n tokens multiplies a one-sided error of a by n (a decay taken from expf was off
// by 4e-5 after 10^4 tokens).  Below -88 (where 2^k becomes 0) the decay is exactly 0.
// x is brought to -88 in place: log a times a gradient that holds a factor a is then 0 there, not NaN.
struct Decay { float a, e; };
__device__ __forceinline__ float power_of_two(float t) {           // 2^k, k in the low bits of t = 1.5 * 2^23 + k
    return __int_as_float((__float_as_int(t) << 23) + 0x3f800000);
}
__device__ __forceinline__ Decay decay(float& x) {
    x = max_nan(x, -88.f);
    const float t = fmaf(x, kLog2e, 12582912.f);
    const float k = t - 12582912.f;
    const float r = fmaf(k, 2.1219444e-4f, fmaf(k, -0.693359375f, x));
    float q = fmaf(r, 1.3950337e-3f, 8.3688218e-3f);
    q = fmaf(q, r, 4.1666210e-2f);
    q = fmaf(q, r, 1.6666520e-1f);
    q = fmaf(q, r, 0.5f);
    const float p = fmaf(r * r, q, r);
    const float sc = power_of_two(t);
    return {fmaf(sc, p, sc), fmaf(sc, p, sc - 1.f)};
}
__device__ __forceinline__ void decay(float& x0, float& x1, Decay& d0, Decay& d1) {
    x0 = max_nan(x0, -88.f);
    x1 = max_nan(x1, -88.f);
    const f2 x = pack(x0, x1), t = fma2(x, both_of(kLog2e), both_of(12582912.f)), k = add2(t, both_of(-12582912.f));
    const f2 r = fma2(k, both_of(2.1219444e-4f), fma2(k, both_of(-0.693359375f), x));
    f2 q = fma2(r, both_of(1.3950337e-3f), both_of(8.3688218e-3f));
    q = fma2(q, r, both_of(4.1666210e-2f));
    q = fma2(q, r, both_of(1.6666520e-1f));
    q = fma2(q, r, both_of(0.5f));
    const f2 p = fma2(mul2(r, r), q, r);
    float t0, t1;
    unpack(t, t0, t1);
    const f2 sc = pack(power_of_two(t0), power_of_two(t1));
    unpack(fma2(sc, p, sc), d0.a, d1.a);
    unpack(fma2(sc, p, add2(sc, both_of(-1.f))), d0.e, d1.e);
}

// exp(-|z|) carries both softplus and sigma.  log1p(q) = q P(q) on [0, 1], off by less than 2^-23.9 of itself.
// It is the square of its root, which is a normal number down to z = -174: a subnormal exp(-|z|) still makes 1 - a^2 and the
// gates' gradients what they are.
__device__ __forceinline__ float tail_root(float z) { return ex2(fabsf(z) * (-0.5f * kLog2e)); }
__device__ __forceinline__ float tail(float z) {
    const float h = tail_root(z);
    return h * h;
}
__device__ __forceinline__ float softplus(float z, float q) {
    float s = fmaf(q, 5.3840620e-3f, -3.0110965e-2f);
    s = fmaf(s, q, 7.9210736e-2f);
    s = fmaf(s, q, -1.3746622e-1f);
    s = fmaf(s, q, 1.9145116e-1f);
    s = fmaf(s, q, -2.4852946e-1f);
    s = fmaf(s, q, 3.3320343e-1f);
    s = fmaf(s, q, -4.9999553e-1f);
    s = fmaf(s, q, 1.f);
    return fmaf(s, q, fmaxf(z, 0.f));
}
// of two logits, times nA
__device__ __forceinline__ void softplus(float z0, float z1, float nA0, float nA1, float& r0, float& r1) {
    const f2 h = pack(tail_root(z0), tail_root(z1)), q = mul2(h, h);
    f2 s = fma2(q, both_of(5.3840620e-3f), both_of(-3.0110965e-2f));
    s = fma2(s, q, both_of(7.9210736e-2f));
    s = fma2(s, q, both_of(-1.3746622e-1f));
    s = fma2(s, q, both_of(1.9145116e-1f));
    s = fma2(s, q, both_of(-2.4852946e-1f));
    s = fma2(s, q, both_of(3.3320343e-1f));
    s = fma2(s, q, both_of(-4.9999553e-1f));
    s = fma2(s, q, both_of(1.f));
    unpack(mul2(fma2(s, q, pack(fmaxf(z0, 0.f), fmaxf(z1, 0.f))), pack(nA0, nA1)), r0, r1);
}
__device__ __forceinline__ float sigmoid(float z, float q) { return (z < 0.f ? q : 1.f) * rcp(1.f + q); }
__device__ __forceinline__ float sigmoid(float z) { return rcp(1.f + ex2(z * -kLog2e)); }

// The input factor s = sqrt(1 - a^2) (0 for a decay above 1).  A log a that is a subnormal number leaves 1 - a^2 one too, while
// s (about 1e-20) and 1 / s are not; so 1 - a^2 is taken times 2^64, past the flushing of the approximations, and s times 2^32.
// Two elements to an instruction where there are two (65,536 packed tokens x 4096 channels forward: 749 us; one by one 823).
constexpr float kFactor = 0x1p32f;
__device__ __forceinline__ void input_powers(float* power, const Decay& d) {      // 2^64 (1 - a^2) = -2^64 e (2 + e)
    power[0] = fmaxf(d.e * fmaf(d.e, -kFactor * kFactor, -2.f * kFactor * kFactor), 0.f);
}
__device__ __forceinline__ void input_powers(float* power, const Decay& d0, const Decay& d1) {
    const f2 e = pack(d0.e, d1.e);
    unpack(mul2(e, fma2(e, both_of(-kFactor * kFactor), both_of(-2.f * kFactor * kFactor))), power[0], power[1]);
    power[0] = fmaxf(power[0], 0.f);
    power[1] = fmaxf(power[1], 0.f);
}
// u times s
template <int N>
__device__ __forceinline__ void times_factors(float* u, const float* power) {
    if constexpr (N == 2) {
        const f2 s = mul2(pack(root(power[0]), root(power[1])), both_of(1.f / kFactor));
        unpack(mul2(pack(u[0], u[1]), s), u[0], u[1]);
    } else {
        u[0] *= root(power[0]) * (1.f / kFactor);
    }
}

}  // namespace glr
}  // namespace gdn
