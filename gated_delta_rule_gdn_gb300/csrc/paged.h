// Requests of the paged key-value cache: appending to it and attention over it, already validated by paged_api.cu.
#pragma once

#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace gdn {

// Keys, or values: [pages][slots][heads][d] with strides in elements, the channels contiguous.
struct PagedSide {
    void* p;
    int64_t page, slot, head;
};
// Token t of sequence n lies in slot t % page_size of page table[n * table_ld + t / page_size].  An entry outside [0, n_pages)
// is no page: nothing is written there, and attention passes over its keys.
struct PagedCache {
    PagedSide k, v;
    const int32_t* table;
    int64_t table_ld;
    int max_pages, page_size, n_pages;
    const int32_t* lengths;     // tokens of each sequence, the call's new ones among them
    int N, Hk, d;
    int bf16;
};

struct PagedAppendArgs {
    PagedCache c;
    const void *k, *v, *q;      // [n_tokens, heads, d] with strides; q or nullptr
    int64_t k_tok, k_head, v_tok, v_head, q_tok, q_head;
    int Hq;
    int64_t n_tokens;
    const int32_t* cu;          // [N + 1] offsets of each sequence's new tokens, or nullptr: one each
    const float *cos, *sin;     // [n_pos, rot / 2]
    int n_pos, rot, interleaved;
    void* q_out;                // [n_tokens, Hq, d] contiguous
};
cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t s);

struct PagedAttnArgs {
    PagedCache c;
    const void* q;              // [N, Hq, d] with strides
    int64_t q_tok, q_head;
    int Hq;
    float scale;
    void* o;                    // [N, Hq, d] contiguous
    float* lse;                 // [N, Hq] or nullptr
    int splits;                 // parts that a sequence's tokens are divided into at most (paged_attn_splits)
    void* ws;
};
int paged_attn_splits(const PagedAttnArgs& a);
// Tokens of one part of a sequence of `len` (2^31 - 256 at most, a multiple of 64 of at least 128), the parts that it has, no more than
// `splits`, and where one begins (the end of the sequence where there is none).  Written so that no sum passes 31 bits.
__host__ __device__ inline int paged_attn_part_tokens(int len, int splits) {
    const int per = len / splits + (len % splits != 0);
    return per <= 128 ? 128 : (per + 63) / 64 * 64;
}
__host__ __device__ inline int paged_attn_parts(int len, int per) { return len / per + (len % per != 0); }
__host__ __device__ inline int paged_attn_part_begin(int len, int per, int split) {
    const int64_t at = (int64_t)per * split;
    return at < len ? (int)at : len;
}
// The workspace, where sequences have several parts: (maximum, sum) of each (sequence, query head, part), read as pairs and so
// first, on the workspace's own alignment; then the parts' d channels, whose number may be odd.
__host__ __device__ inline int64_t paged_attn_tops_at(const PagedAttnArgs& a, int n, int hq, int split) {      // in floats
    return (((int64_t)n * a.Hq + hq) * a.splits + split) * 2;
}
__host__ __device__ inline int64_t paged_attn_sums_at(const PagedAttnArgs& a, int n, int hq, int split) {
    return (int64_t)a.c.N * a.Hq * a.splits * 2 + (((int64_t)n * a.Hq + hq) * a.splits + split) * a.c.d;
}
inline size_t paged_attn_workspace_bytes(const PagedAttnArgs& a) {
    return a.splits <= 1 ? 0 : sizeof(float) * (size_t)paged_attn_sums_at(a, a.c.N, 0, 0);
}
cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t s);

}  // namespace gdn
