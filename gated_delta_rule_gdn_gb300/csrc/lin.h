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
    // Backward, the parts of the decays' gradient, each [block of columns][h][token] (x has dc columns):
    LinTok x;
    float* dots;            // x_i . (s_inter a_i S), or nullptr
    float* pair_dots;       // x_i . (the sum over j) without j = i (the generic walk), or nullptr
    // States at the starts of spans of kLinSpan tokens, [span slot][h][block][da][block's columns]: the forward walk writes
    // them, the reverse one writes anchors[span slot][h][block], e^(G_end) times the inner product with its own state behind
    // the span's first chunk.
    float* spans;
    float* anchors;
    // Segments of a walk (0: none) of seg_chunks kLinChunk tokens: [segment slot][h][block] states (128 x kLinCols on the tensor cores,
    // else da x kLinGenericCols), first of each segment from nothing, then entering it, and [segment slot][h] the log (base 2) of what each keeps of the state entering it.
    int seg_chunks;
    float *seg_states, *seg_kept;
    int test_stall;         // test of the bounded waits: the copies of c are left out
    int fine;               // scaled values of the state as three bf16 numbers instead of two (walks that sum up a constant decay's gradient)
    int wait_first;         // the kernel before it has to be complete (walks are launched before it is)
    __host__ __device__ int N() const { return cu ? n_seqs : B; }
    __host__ __device__ int64_t rows() const { return (int64_t)B * T; }
};
// A span is a chunk of the tensor cores, so that no inner product is carried from one to the next there, where each adds its rounding;
// the price is 512 bytes of states a token and head (128 x 128) to write and to read.
constexpr int kLinSpan = 128, kLinGenericChunk = 32, kLinChunk = 128;
// The span slots of a call: those of sequence n begin at first_token / kLinSpan + n.
inline int64_t lin_slots(int64_t rows, int64_t N, int64_t size) { return rows / size + N + 1; }
// Segments of `size` tokens of a sequence of `len` (size + len may pass 31 bits).
__host__ __device__ inline int lin_segments(int len, int size) { return len / size + (len % size != 0); }
inline int64_t lin_span_slots(int64_t rows, int64_t N) { return lin_slots(rows, N, kLinSpan); }
// Columns of c that a block of threads takes (the generic walk, the tensor-core one), for dots and anchors.
constexpr int kLinGenericCols = 32, kLinCols = 64;
inline int lin_blocks(int dc, bool tensor) { return (dc + (tensor ? kLinCols : kLinGenericCols) - 1) / (tensor ? kLinCols : kLinGenericCols); }
inline size_t lin_span_floats(int da, int dc, bool tensor) {
    return tensor ? (size_t)128 * kLinCols * lin_blocks(dc, true) : (size_t)da * kLinGenericCols * lin_blocks(dc, false);
}

// The tensor-core walk and the generic one: whether the former takes the request, chunks of kLinChunk tokens of a segment of either
// (0: none), and the walks.  The former's dots are those of the state's part alone.
bool lin_tensor_fits(const LinWalk& w);
int lin_segment_chunks(int64_t rows, int64_t N, bool packed, int H, int da, int dc, bool tensor);
// behind: launched while the stream's last kernel still runs (one of this operator, which does not complete before those before it).  A walk that reads nothing of what came before runs at once on the SMs that are free; with spans, or in
// segments, it waits.
cudaError_t launch_lin_walk_tensor(const LinWalk& w, bool behind, cudaStream_t s);
cudaError_t launch_lin_walk_generic(const LinWalk& w, bool behind, cudaStream_t s);
cudaError_t launch_lin_segments(const LinWalk& w, cudaStream_t s);
// What the pairs of tokens of a chunk have of the decays' gradient, pairs[h][token]: the sum over the keys before the token
// minus the sum over the queries behind it, of scale e^(G_i - G_j) (q_i . k_j) (dO_i . v_j).
struct LinPairs {
    LinTok q, k, v, o;
    int dk, dv;
    float scale;
    const float* g;
    int64_t g_tok, g_head;
    const int32_t* cu;
    int n_seqs, B, T, H;
    float* pairs;
    __host__ __device__ int N() const { return cu ? n_seqs : B; }
    __host__ __device__ int64_t rows() const { return (int64_t)B * T; }
};
cudaError_t launch_lin_pairs(const LinPairs& a, cudaStream_t s);
cudaError_t lin_pairs_read_and_clear_status(unsigned* value, bool clear);
cudaError_t lin_read_and_clear_status(unsigned* value, bool clear);

// dg from the walks' parts.  With S_in the state entering a token's chunk and D_out the gradient of the state leaving it,
//     dg_t = sum over pairs j < t <= i of the chunk  +  sum_{i >= t} plus_i  +  sum_{j < t} minus_j  +  e^(G_end) <D_out, S_in>
// where plus_i = q_i . (the part of dq_i that S_in has), minus_j = k_j . (the part of dk_j that D_out has), and the pairs are
// sum_{i >= t} (pairs_i - pairs_minus_i), i over the chunk, of the sums over keys before i and over queries behind i.  No two
// of the four cancel.  The last is an inner product at a span's first chunk (anchors) and goes on from chunk to chunk by
//     <D, S> at their border = the former's minus and last = the latter's plus and last.
// With per_head, dg is [H], the sum over all tokens, by way of `part` [span slots][H].
struct LinDg {
    const float *plus, *minus, *pairs, *pairs_minus, *anchors;
    int blocks, pair_blocks, anchor_blocks, chunk;     // (pairs_minus nullptr: in pairs)
    float* dg;
    int per_head;
    float* part;
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
