// Short causal depthwise convolution with its activation, its gradients, and the decode step.
//   p_t = b + sum_j w_j x_{t - W + 1 + j},  y_t = silu(p_t) or p_t; inputs before a sequence's first token are its
//   initial state (its last W - 1 inputs, oldest first) or zero.
// Backward: ds = dy silu'(p), dx_t = sum_j w_j ds_{t + W - 1 - j}, dw_j = sum_t ds_t x_{t - W + 1 + j}, db = sum ds.

#include "mixer.h"
#include "mixer_common.cuh"

namespace gdn {
namespace {

using mix::bf16;
using mix::ld;
using mix::st;

// the input at place `at` of sequence n (negative: the initial state), channel c
template <typename T>
__device__ __forceinline__ float input(const ConvArgs& a, int64_t row0, int n, int at, int c) {
    if (at >= 0) return ld(static_cast<const T*>(a.x) + (row0 + at) * a.ldx + c);
    return a.h0 ? ld(static_cast<const T*>(a.h0) + ((int64_t)n * (a.W - 1) + at + a.W - 1) * a.D + c) : 0.f;
}

template <typename T>
__device__ __forceinline__ float pre(const ConvArgs& a, int64_t row0, int n, int at, int c) {
    float p = a.b ? a.b[c] : 0.f;
    for (int j = 0; j < a.W; ++j) p = fmaf(a.w[(size_t)c * a.W + j], input<T>(a, row0, n, at - a.W + 1 + j, c), p);
    return p;
}
__device__ __forceinline__ float act(const ConvArgs& a, float p) { return a.silu ? p / (1.f + expf(-p)) : p; }

// the gradient of p at place `at` < len
template <typename T>
__device__ __forceinline__ float grad_pre(const ConvArgs& a, int64_t row0, int n, int at, int c) {
    const float dy = ld(static_cast<const T*>(a.dy) + (row0 + at) * a.D + c);
    if (!a.silu) return dy;
    const float p = pre<T>(a, row0, n, at, c), sg = 1.f / (1.f + expf(-p));
    return dy * sg * (1.f + p * (1.f - sg));
}

// the gradient of the input at place `at` (negative: the initial state's)
template <typename T>
__device__ __forceinline__ float grad_in(const ConvArgs& a, int64_t row0, int n, int len, int at, int c) {
    float s = 0.f;
    for (int j = 0; j < a.W; ++j) {
        const int t = at + a.W - 1 - j;
        if (t >= 0 && t < len) s = fmaf(a.w[(size_t)c * a.W + j], grad_pre<T>(a, row0, n, t, c), s);
    }
    const int tail = at - (len - (a.W - 1));        // its place in the final state
    if (a.dhT && tail >= 0) s += ld(static_cast<const T*>(a.dhT) + ((int64_t)n * (a.W - 1) + tail) * a.D + c);
    return s;
}

__device__ __forceinline__ void token(const ConvArgs& a, int64_t r, int64_t* row0, int* n, int* at, int* len) {
    const int b = (int)(r / a.T), t = (int)(r % a.T);
    if (a.cu) {
        const mix::Span s = mix::span_of(a.cu, a.n_seqs, a.T, t);
        *row0 = s.first;
        *n = s.n;
        *at = t - s.first;
        *len = s.end - s.first;
    } else {
        *row0 = (int64_t)b * a.T;
        *n = b;
        *at = t;
        *len = a.T;
    }
}
__device__ __forceinline__ void sequence(const ConvArgs& a, int n, int64_t* row0, int* len) {
    *row0 = a.cu ? mix::clamp_off(a.cu[n], a.T) : (int64_t)n * a.T;
    *len = a.cu ? max(mix::clamp_off(a.cu[n + 1], a.T) - (int)*row0, 0) : a.T;
}

template <typename T>
__global__ void conv_fwd_kernel(const ConvArgs a) {
    const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, r = id / a.D;
    const int c = (int)(id % a.D);
    if (r >= (int64_t)a.B * a.T) return;
    int64_t row0;
    int n, at, len;
    token(a, r, &row0, &n, &at, &len);
    st(static_cast<T*>(a.y) + r * a.D + c, act(a, pre<T>(a, row0, n, at, c)));
}

// the last W - 1 inputs of every sequence (forward), and the gradients of the initial ones (backward)
template <typename T>
__global__ void conv_state_kernel(const ConvArgs a) {
    const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, r = id / a.D;
    const int c = (int)(id % a.D);
    if (r >= (int64_t)a.N() * (a.W - 1)) return;
    const int n = (int)(r / (a.W - 1)), j = (int)(r % (a.W - 1));
    int64_t row0;
    int len;
    sequence(a, n, &row0, &len);
    if (a.hT) st(static_cast<T*>(a.hT) + r * a.D + c, input<T>(a, row0, n, len - (a.W - 1) + j, c));
    if (a.dh0) st(static_cast<T*>(a.dh0) + r * a.D + c, grad_in<T>(a, row0, n, len, j - (a.W - 1), c));
}

template <typename T>
__global__ void conv_bwd_kernel(const ConvArgs a) {
    const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, r = id / a.D;
    const int c = (int)(id % a.D);
    if (r >= (int64_t)a.B * a.T) return;
    int64_t row0;
    int n, at, len;
    token(a, r, &row0, &n, &at, &len);
    st(static_cast<T*>(a.dx) + r * a.D + c, grad_in<T>(a, row0, n, len, at, c));
}

constexpr int kRowsPerPart = 128;

// weight gradients of kRowsPerPart tokens of a channel: [W] then the bias's
template <typename T>
__global__ void conv_dw_kernel(const ConvArgs a, float* part) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= a.D) return;
    float s[5] = {};
    const int64_t lo = (int64_t)blockIdx.y * kRowsPerPart, rows = (int64_t)a.B * a.T;
    for (int64_t r = lo; r < min(lo + kRowsPerPart, rows); ++r) {
        int64_t row0;
        int n, at, len;
        token(a, r, &row0, &n, &at, &len);
        const float g = grad_pre<T>(a, row0, n, at, c);
        for (int j = 0; j < a.W; ++j) s[j] = fmaf(g, input<T>(a, row0, n, at - a.W + 1 + j, c), s[j]);
        s[4] += g;
    }
    for (int j = 0; j < 5; ++j) part[((size_t)blockIdx.y * 5 + j) * a.D + c] = s[j];
}

__global__ void conv_param_kernel(const ConvArgs a, const float* part, int parts) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= a.D) return;
    float s[5] = {};
    for (int k = 0; k < parts; ++k)
        for (int j = 0; j < 5; ++j) s[j] += part[((size_t)k * 5 + j) * a.D + c];
    for (int j = 0; j < a.W; ++j) a.dw[(size_t)c * a.W + j] = s[j];
    if (a.db) a.db[c] = s[4];
}

template <typename T>
__global__ void conv_step_kernel(const ConvArgs a, const T* state, T* out) {
    const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, n = id / a.D;
    const int c = (int)(id % a.D);
    if (n >= a.B) return;
    const T* h = state + n * (a.W - 1) * a.D + c;
    T* o = out + n * (a.W - 1) * a.D + c;
    const T x = static_cast<const T*>(a.x)[n * a.ldx + c];
    float p = a.b ? a.b[c] : 0.f;
    for (int j = 0; j < a.W - 1; ++j) {
        const T v = h[(int64_t)j * a.D];
        p = fmaf(a.w[(size_t)c * a.W + j], ld(&v), p);
        if (j > 0) o[(int64_t)(j - 1) * a.D] = v;
    }
    p = fmaf(a.w[(size_t)c * a.W + a.W - 1], ld(&x), p);
    o[(int64_t)(a.W - 2) * a.D] = x;
    st(static_cast<T*>(a.y) + n * a.D + c, act(a, p));
}

// (grid.y of the weight gradients: up to 65,535 parts, 8M tokens; mixer_api.cu refuses more)
unsigned blocks_for(int64_t n) { return (unsigned)((n + 127) / 128); }
int parts_of(const ConvArgs& a) { return (int)(((int64_t)a.B * a.T + kRowsPerPart - 1) / kRowsPerPart); }

template <typename T>
cudaError_t fwd(const ConvArgs& a, cudaStream_t s) {
    const int64_t rows = (int64_t)a.B * a.T;
    if (rows > 0) conv_fwd_kernel<T><<<blocks_for(rows * a.D), 128, 0, s>>>(a);
    if (a.hT) conv_state_kernel<T><<<blocks_for((int64_t)a.N() * (a.W - 1) * a.D), 128, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t bwd(const ConvArgs& a, cudaStream_t s) {
    const int64_t rows = (int64_t)a.B * a.T;
    float* part = static_cast<float*>(a.ws);
    if (rows > 0) {
        conv_bwd_kernel<T><<<blocks_for(rows * a.D), 128, 0, s>>>(a);
        conv_dw_kernel<T><<<dim3((a.D + 127) / 128, parts_of(a)), 128, 0, s>>>(a, part);
    }
    conv_param_kernel<<<(a.D + 127) / 128, 128, 0, s>>>(a, part, parts_of(a));
    if (a.dh0) conv_state_kernel<T><<<blocks_for((int64_t)a.N() * (a.W - 1) * a.D), 128, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t conv_workspace_bytes(const ConvArgs& a) { return (size_t)parts_of(a) * 5 * a.D * sizeof(float); }
cudaError_t launch_conv_fwd(const ConvArgs& a, cudaStream_t s) { return a.bf16 ? fwd<bf16>(a, s) : fwd<float>(a, s); }
cudaError_t launch_conv_bwd(const ConvArgs& a, cudaStream_t s) { return a.bf16 ? bwd<bf16>(a, s) : bwd<float>(a, s); }

cudaError_t launch_conv_step(const ConvArgs& a, const void* state, void* state_out, cudaStream_t s) {
    const unsigned blocks = blocks_for((int64_t)a.B * a.D);
    if (a.bf16)
        conv_step_kernel<bf16><<<blocks, 128, 0, s>>>(a, static_cast<const bf16*>(state), static_cast<bf16*>(state_out));
    else
        conv_step_kernel<float><<<blocks, 128, 0, s>>>(a, static_cast<const float*>(state),
                                                       static_cast<float*>(state_out));
    return cudaGetLastError();
}

}  // namespace gdn
