// Requests of the operators around the delta rule, already validated by mixer_api.cu: the gated linear recurrence
// (glr_scan.cu), the query/key head norm with rotation (qk_norm.cu) and the short convolution (short_conv.cu).
#pragma once

#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace gdn {

// Gated linear recurrence.  Rows of x, g and gi are ld_* elements apart; every other tensor is contiguous.
struct GlrArgs {
    const void* x;          // [B, T, D]
    const void* g;          // [B, T, D]
    const void* gi;         // [B, T, D] input-gate logits or nullptr
    const float* A_log;     // [D] or nullptr (g is log a)
    const float* dt_bias;   // [D] or nullptr
    int normalize;
    const float* h0;        // [N, D] or nullptr
    float* hT;              // [N, D] or nullptr
    const int32_t* cu;      // [n_seqs + 1] device or nullptr
    int n_seqs;
    void* o;                // [B, T, D], or nullptr (checkpoints only)
    float* ckpt;            // [B, ceil(T / 64), D]: the state before tokens 0, 64, 128, ... of a row, or nullptr
    // backward
    const void* dO;         // [B, T, D]
    const float* dhT;       // [N, D] or nullptr
    void* dx;               // [B, T, D]
    void* dg;               // [B, T, D]
    void* di;               // [B, T, D] (with gi)
    float* dh0;             // [N, D] or nullptr
    float* dA;              // [D] (with A_log)
    float* ddt;             // [D] or nullptr
    void* ws;
    int B, T, D;
    int64_t ldx, ldg, ldi;
    int bf16, g_bf16;       // element types: x, gi, o, dO, dx, di; g, dg
    int test_stall;         // test of the bounded waits: the first tile of every row keeps its map to itself
    __host__ __device__ int N() const { return cu ? n_seqs : B; }
};
constexpr int kGlrTile = 64;   // tokens between checkpoints
size_t glr_workspace_bytes(const GlrArgs& a, bool backward);
bool glr_vector(const GlrArgs& a, int V);      // rows can be read and written V channels at a time
cudaError_t glr_read_and_clear_status(unsigned* value, bool clear);
cudaError_t glr_bwd_read_and_clear_status(unsigned* value, bool clear);
cudaError_t launch_glr_fwd(const GlrArgs& a, cudaStream_t s);
cudaError_t launch_glr_bwd(const GlrArgs& a, cudaStream_t s);

struct GlrStepArgs {
    const void* x;
    const void* g;
    const void* gi;
    const float* A_log;
    const float* dt_bias;
    int normalize;
    const float* h;         // [N, D]
    float* h_out;           // [N, D], h itself or another buffer
    void* o;                // [N, D]
    int N, D;
    int64_t ldx, ldg, ldi;
    int bf16, g_bf16;
};
cudaError_t launch_glr_step(const GlrStepArgs& a, cudaStream_t s);

// Query/key head norm with rotation.
struct QkNormArgs {
    const void* in[2];      // q [n, Hq, d] and k [n, Hk, d] with token and head strides
    const void* dout[2];    // backward: gradients of the outputs, contiguous
    void* out[2];           // forward: outputs; backward: gradients of the inputs; contiguous
    const float* w[2];      // [d] or nullptr
    float* dw[2];           // backward: [d] or nullptr
    int64_t tok_stride[2], head_stride[2];
    int H[2];
    int64_t n;              // tokens
    int T;                  // tokens of a sequence (the position without `pos` is the token's index in it)
    int d;
    float c, eps;           // 1/d (rms) or 1 (l2)
    const float* cos;       // [n_pos, rot / 2]
    const float* sin;
    int n_pos, rot, interleaved;
    const int32_t* pos;     // [n] or nullptr
    int bf16;
    void* ws;
};
size_t qk_norm_workspace_bytes(const QkNormArgs& a);
cudaError_t launch_qk_norm_fwd(const QkNormArgs& a, cudaStream_t s);
cudaError_t launch_qk_norm_bwd(const QkNormArgs& a, cudaStream_t s);

// Short causal depthwise convolution.
struct ConvArgs {
    const void* x;          // [B, T, D], rows ldx elements apart
    const float* w;         // [D, W]
    const float* b;         // [D] or nullptr
    int silu;
    const void* h0;         // [N, W - 1, D] or nullptr
    void* hT;               // [N, W - 1, D] or nullptr
    const int32_t* cu;
    int n_seqs;
    void* y;                // [B, T, D]
    // backward
    const void* dy;         // [B, T, D]
    const void* dhT;        // [N, W - 1, D] or nullptr
    void* dx;               // [B, T, D]
    float* dw;              // [D, W]
    float* db;              // [D] or nullptr
    void* dh0;              // [N, W - 1, D] or nullptr
    void* ws;
    int B, T, D, W;
    int64_t ldx;
    int bf16;
    __host__ __device__ int N() const { return cu ? n_seqs : B; }
};
size_t conv_workspace_bytes(const ConvArgs& a);
cudaError_t launch_conv_fwd(const ConvArgs& a, cudaStream_t s);
cudaError_t launch_conv_bwd(const ConvArgs& a, cudaStream_t s);
cudaError_t launch_conv_step(const ConvArgs& a, const void* state, void* state_out, cudaStream_t s);

}  // namespace gdn
