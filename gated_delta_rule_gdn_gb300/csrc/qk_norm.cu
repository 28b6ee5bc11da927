// Norm of every query and key head with the position rotation in the same pass, and its gradients.
//   y = w x r,  r = 1 / sqrt(c sum x^2 + eps)  (c = 1/d: root mean square; c = 1: unit length)
//   the first `rot` channels of y turn by the angles of the token's position: pairs (i, i + rot/2), or (2i, 2i + 1)
//   interleaved.
// Backward: dy = the output's gradient turned back, dw = sum dy x r, e = w dy, dx = r (e - c r^2 x sum(x e)).

#include <type_traits>

#include "mixer.h"
#include "mixer_common.cuh"

namespace gdn {
namespace {

using mix::bf16;
using mix::ld;
using mix::st;

__device__ __forceinline__ float warp_sum(float v) {
    for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// partner channel, its sign in the forward rotation, and the angle index of rotated channel j
__device__ __forceinline__ void pair_of(const QkNormArgs& a, int j, int* other, float* sign, int* angle) {
    if (a.interleaved) {
        *other = j ^ 1;
        *sign = (j & 1) ? 1.f : -1.f;
        *angle = j >> 1;
    } else {
        const int half = a.rot >> 1;
        *other = j < half ? j + half : j - half;
        *sign = j < half ? -1.f : 1.f;
        *angle = j < half ? j : j - half;
    }
}

constexpr int kMaxD = 256, kWarps = 4;

__device__ __forceinline__ int position(const QkNormArgs& a, int64_t tok) {
    const int p = a.pos ? a.pos[tok] : (int)(tok % a.T);
    return min(max(p, 0), a.n_pos - 1);
}

// one warp per (token, head)
template <typename T>
__global__ void qk_fwd_kernel(const QkNormArgs a) {
    __shared__ float buf[kWarps][kMaxD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t id = (int64_t)blockIdx.x * kWarps + warp;
    const int heads = a.H[0] + a.H[1];
    const int64_t tok = id / heads;
    const int hh = (int)(id % heads), which = hh >= a.H[0], h = which ? hh - a.H[0] : hh;
    if (tok >= a.n) return;
    const T* x = static_cast<const T*>(a.in[which]) + tok * a.tok_stride[which] + h * a.head_stride[which];
    T* y = static_cast<T*>(a.out[which]) + (tok * a.H[which] + h) * a.d;
    float ss = 0.f;
    for (int j = lane; j < a.d; j += 32) {
        const float v = ld(x + j);
        ss = fmaf(v, v, ss);
    }
    const float r = rsqrtf(fmaf(a.c, warp_sum(ss), a.eps));
    for (int j = lane; j < a.d; j += 32) buf[warp][j] = ld(x + j) * r * (a.w[which] ? a.w[which][j] : 1.f);
    __syncwarp();
    const int p = a.rot ? position(a, tok) : 0;
    for (int j = lane; j < a.d; j += 32) {
        float v = buf[warp][j];
        if (j < a.rot) {
            int o, k;
            float sg;
            pair_of(a, j, &o, &sg, &k);
            const int64_t at = (int64_t)p * (a.rot >> 1) + k;
            v = v * a.cos[at] + sg * buf[warp][o] * a.sin[at];
        }
        st(y + j, v);
    }
}

// one warp per (token, head); the block's weight gradients go to a partial row each
template <typename T>
__global__ void qk_bwd_kernel(const QkNormArgs a, float* part) {
    __shared__ float buf[kWarps][kMaxD];
    __shared__ float dw[2][kMaxD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int heads = a.H[0] + a.H[1];
    float acc[2][kMaxD / 32] = {};
    for (int64_t id = (int64_t)blockIdx.x * kWarps + warp; id < a.n * heads; id += (int64_t)gridDim.x * kWarps) {
        const int64_t tok = id / heads;
        const int hh = (int)(id % heads), which = hh >= a.H[0], h = which ? hh - a.H[0] : hh;
        const T* x = static_cast<const T*>(a.in[which]) + tok * a.tok_stride[which] + h * a.head_stride[which];
        const T* dz = static_cast<const T*>(a.dout[which]) + (tok * a.H[which] + h) * a.d;
        T* dx = static_cast<T*>(a.out[which]) + (tok * a.H[which] + h) * a.d;
        const int p = a.rot ? position(a, tok) : 0;
        __syncwarp();
        for (int j = lane; j < a.d; j += 32) buf[warp][j] = ld(dz + j);
        __syncwarp();
        float ss = 0.f, xe = 0.f, e[kMaxD / 32], xv[kMaxD / 32];
#pragma unroll
        for (int i = 0; i < kMaxD / 32; ++i) {
            const int j = lane + 32 * i;
            e[i] = xv[i] = 0.f;
            if (j >= a.d) continue;
            float v = buf[warp][j];
            if (j < a.rot) {
                int o, k;
                float sg;
                pair_of(a, j, &o, &sg, &k);
                const int64_t at = (int64_t)p * (a.rot >> 1) + k;
                v = v * a.cos[at] - sg * buf[warp][o] * a.sin[at];
            }
            xv[i] = ld(x + j);
            ss = fmaf(xv[i], xv[i], ss);
            e[i] = v;
        }
        const float r = rsqrtf(fmaf(a.c, warp_sum(ss), a.eps));
#pragma unroll
        for (int i = 0; i < kMaxD / 32; ++i) {
            const int j = lane + 32 * i;
            if (j >= a.d) continue;
            if (which) acc[1][i] += e[i] * xv[i] * r; else acc[0][i] += e[i] * xv[i] * r;
            if (a.w[which]) e[i] *= a.w[which][j];
            xe = fmaf(xv[i], e[i], xe);
        }
        xe = warp_sum(xe) * a.c * r * r;
#pragma unroll
        for (int i = 0; i < kMaxD / 32; ++i) {
            const int j = lane + 32 * i;
            if (j < a.d) st(dx + j, r * (e[i] - xv[i] * xe));
        }
    }
    for (int w = 0; w < kWarps; ++w) {     // warps in turn: a fixed order
        if (warp == w)
#pragma unroll
            for (int i = 0; i < kMaxD / 32; ++i)
                for (int k = 0; k < 2; ++k) {
                    const int j = lane + 32 * i;
                    dw[k][j] = (w ? dw[k][j] : 0.f) + acc[k][i];
                }
        __syncthreads();
    }
    for (int j = threadIdx.x; j < 2 * a.d; j += blockDim.x)
        part[(size_t)blockIdx.x * 2 * a.d + j] = dw[j / a.d][j % a.d];
}

__global__ void qk_dw_kernel(const float* part, int rows, int d, float* dwq, float* dwk) {
    const int j = blockIdx.x * blockDim.x + threadIdx.x;
    if (j >= 2 * d) return;
    float s = 0.f;
    for (int r = 0; r < rows; ++r) s += part[(size_t)r * 2 * d + j];
    float* out = j < d ? dwq : dwk;
    if (out) out[j % d] = s;
}

int bwd_blocks(const QkNormArgs& a) {
    const int64_t rows = a.n * (a.H[0] + a.H[1]);
    const int64_t want = (rows + kWarps - 1) / kWarps;
    return (int)(want < 152 * 8 ? want : 152 * 8);
}

}  // namespace

size_t qk_norm_workspace_bytes(const QkNormArgs& a) { return (size_t)bwd_blocks(a) * 2 * a.d * sizeof(float); }

cudaError_t launch_qk_norm_fwd(const QkNormArgs& a, cudaStream_t s) {
    const int64_t rows = a.n * (a.H[0] + a.H[1]);
    const unsigned blocks = (unsigned)((rows + kWarps - 1) / kWarps);
    if (a.bf16) qk_fwd_kernel<bf16><<<blocks, kWarps * 32, 0, s>>>(a);
    else qk_fwd_kernel<float><<<blocks, kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_qk_norm_bwd(const QkNormArgs& a, cudaStream_t s) {
    const int blocks = bwd_blocks(a);          // 0 without tokens: the weight gradients are then zero
    float* part = static_cast<float*>(a.ws);
    if (blocks == 0) {}
    else if (a.bf16) qk_bwd_kernel<bf16><<<blocks, kWarps * 32, 0, s>>>(a, part);
    else qk_bwd_kernel<float><<<blocks, kWarps * 32, 0, s>>>(a, part);
    if (a.dw[0] || a.dw[1]) qk_dw_kernel<<<(2 * a.d + 127) / 128, 128, 0, s>>>(part, blocks, a.d, a.dw[0], a.dw[1]);
    return cudaGetLastError();
}

}  // namespace gdn
