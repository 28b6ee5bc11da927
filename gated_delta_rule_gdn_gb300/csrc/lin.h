// Requests of linear attention with a decay for each head, already validated by lin_api.cu.
#pragma once

#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace gdn {

// One of the walk's token inputs: value head h reads head h / group.
struct LinTok {
    const void* p;
    int64_t tok, head;      // strides in elements
    int group;
};

// The one operation behind the forward and all token gradients, a walk over the tokens of every sequence and value head:
//     out_i = s_intra sum_j e^(G_i - G_j) (a_i . b_j) c_j  +  s_inter a_i S,      j <= i (j >= i and e^(G_j - G_i) with rev)
// where S, decayed up to the token, is s_in followed by s_state times the products b_j c_j^T of all tokens before it (behind).
//     forward   a = q,  b = k,  c = v,  S = state
//     dq        a = dO, b = v,  c = k,  S = state^T
//     dk        a = v,  b = dO, c = q,  S = (gradient of the state)^T, rev
//     dv        a = k,  b = q,  c = dO, S = gradient of the state, rev
struct LinWalk {
    LinTok a, b, c;         // widths da, da, dc
    int da, dc;
    int rev;
    float s_intra, s_inter, s_state;
    const float* g;         // log decays, element (token, head) at token * g_tok + head * g_head
    int64_t g_tok, g_head;
    const float* s_in;      // [N, H] states of da * dc elements or nullptr: (r, c) at r * s_r + c * s_c
    float* s_out;           // the state behind the last token (before the first), the same layout, or nullptr
    int s_r, s_c;
    void* out;              // [tokens, H, dc] contiguous, the tokens' type or (out_f32) fp32
    int out_f32;
    const int32_t* cu;
    int n_seqs, B, T, H;
    int bf16;
    // Backward, the parts of the decays' gradient: dots[block][h][token] = x_i . out_i over the block's columns of c, without
    // the pair (i, i).  x has dc columns.
    LinTok x;
    float* dots;            // or nullptr
    // States at the ends of spans of kLinSpan tokens, [span slot][h][block][da][block's columns]: the forward walk writes
    // them, the reverse one writes anchors[span slot][h][block], the inner product of its state with them.
    float* spans;
    float* anchors;
    __host__ __device__ int N() const { return cu ? n_seqs : B; }
    __host__ __device__ int64_t rows() const { return (int64_t)B * T; }
};
constexpr int kLinSpan = 1024;
// The span slots of a call: those of sequence n begin at first_token / kLinSpan + n.
inline int64_t lin_span_slots(int64_t rows, int64_t N) { return rows / kLinSpan + N + 1; }
// Columns of c that a block of threads takes (the generic walk, the tensor-core one), for dots and anchors.
constexpr int kLinGenericCols = 32, kLinCols = 64;
inline int lin_blocks(int dc, bool tensor) { return (dc + (tensor ? kLinCols : kLinGenericCols) - 1) / (tensor ? kLinCols : kLinGenericCols); }
inline size_t lin_span_floats(int da, int dc, bool tensor) {
    return tensor ? (size_t)128 * kLinCols * lin_blocks(dc, true) : (size_t)da * kLinGenericCols * lin_blocks(dc, false);
}

cudaError_t launch_lin_walk_generic(const LinWalk& w, cudaStream_t s);

// dg from the walks' dots and anchors: dg_t = <D, S> at its span's end + sum over the span's tokens i >= t of (q_i . dq_i -
// k_i . dk_i).  With per_head, dg is [H], the sum over all tokens, by way of `part` [span slots][H].
struct LinDg {
    const float *plus, *minus, *anchors;
    int blocks, anchor_blocks;
    float* dg;
    int per_head;
    double* part;
    const int32_t* cu;
    int n_seqs, B, T, H;
    __host__ __device__ int N() const { return cu ? n_seqs : B; }
    __host__ __device__ int64_t rows() const { return (int64_t)B * T; }
};
cudaError_t launch_lin_dg(const LinDg& a, cudaStream_t s);
// out[row, hk] = sum over the group's value heads, in order, of part[row, h] (fp32), d elements each
cudaError_t launch_lin_group_sum(const float* part, void* out, int bf16, int64_t rows, int Hk, int group, int d, cudaStream_t s);

struct LinStepArgs {
    LinTok q, k, v;         // strides over sequences and heads
    const float* g;
    int64_t g_tok, g_head;
    float scale;
    const float* state;     // [N, H, dk, dv]
    float* state_out;       // state itself or another buffer
    void* o;                // [N, H, dv]
    int N, H, dk, dv, bf16;
};
cudaError_t launch_lin_step(const LinStepArgs& a, cudaStream_t s);

}  // namespace gdn
