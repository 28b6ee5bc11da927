// Device pieces shared by the tensor-core kernels of linear attention: packed arithmetic, and one lane that issues.
#pragma once

#include "internal.h"
#include "lin_common.cuh"
#include "tc_common.cuh"

namespace gdn {
namespace {

using namespace tc;
using mix::bf16;

constexpr int CK = kLinChunk;                             // tokens of a chunk
constexpr uint64_t kWait = 2000000000ull;
using lin::last_behind;

__device__ __forceinline__ uint32_t bf2(float x, float y) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float finite_or_0(float x) { return fabsf(x) < INFINITY ? x : 0.f; }
__device__ __forceinline__ float ex2(float x) {           // 2^x to 2^-22; 0 below 2^-126
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// two at a time
struct F2 { float x, y; };
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 d;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 d;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
// One lane of a converged warp.  (Products issued from a branch that the compiler knows to be one lane's take their operands
// from the warp's registers, one in 33 to 64 cycles as the tensor cores take them; behind `lane == 0` inside the loop 70 to 150.)
__device__ __forceinline__ bool elected() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}
// Column sums of a 32 x 32 block, a row a lane: lane l gets that of column l.
__device__ __forceinline__ float column_sums(float (&v)[32], int lane) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1)
#pragma unroll
        for (int k = 0; k < s; ++k) {
            const float send = lane & s ? v[k] : v[k + s], keep = lane & s ? v[k + s] : v[k];
            v[k] = keep + __shfl_xor_sync(0xffffffffu, send, s);
        }
    return v[0];
}

// [tokens, heads, d] bf16 with strides: boxes of 64 channels x 1 head x 128 tokens
inline bool token_map(CUtensorMap* m, const LinTok& t, int d, int heads, int64_t rows) {
    return make_map_strided(m, t.p, rows, heads, d, t.tok, t.head, CK);
}

}  // namespace
}  // namespace gdn
