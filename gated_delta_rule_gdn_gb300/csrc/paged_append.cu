// Appending keys and values to a paged cache, with the position rotation of keys (and queries) on the way.
//
// One block takes one new token: all its key, value and query heads, in vectors of 16 bytes (a rotated item is the two vectors
// whose channels turn with one another, or one vector of interleaved pairs).  Each value is read and written once, so the bound
// is memory, or for a decode step the chain from the length over the table to the store, which is one look-up for the block
// while its inputs are on the way.

#include "mixer_common.cuh"
#include "paged.h"

namespace gdn {
namespace {

using mix::bf16;

// The sequence of token t: the last n with cu[n] <= t, 32 candidates at a time (all lanes of a warp call it).
__device__ __forceinline__ int sequence_of(const int32_t* cu, int N, int64_t t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = N;
    while (n > 1) {
        const int step = (n + 31) / 32, at = lane * step;
        const unsigned below = __ballot_sync(0xffffffffu, at < n && (at == 0 || cu[lo + at] <= t));
        const int hit = 31 - __clz(below);
        lo += hit * step;
        n = min(step, n - hit * step);
    }
    return lo;
}

template <typename T, int V>
__global__ void __launch_bounds__(256) paged_append_kernel(const PagedAppendArgs a) {
    using Vec = mix::Vec<T, V>;
    const PagedCache& c = a.c;
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x;
    int n;
    int64_t pos;
    if (a.cu) {
        n = sequence_of(a.cu, c.N, t);
        if (t < a.cu[n] || t >= a.cu[n + 1]) return;       // a row behind the last sequence
        pos = (int64_t)c.lengths[n] - ((int64_t)a.cu[n + 1] - t);
    } else {
        n = (int)t;
        pos = (int64_t)c.lengths[n] - 1;
    }
    int64_t k_at = -1, v_at = 0;                           // offsets of the token's slot
    if (pos >= 0 && pos / c.page_size < c.max_pages) {
        const int page = c.table[n * c.table_ld + pos / c.page_size];
        if (page >= 0 && page < c.n_pages) {
            k_at = page * c.k.page + pos % c.page_size * c.k.slot;
            v_at = page * c.v.page + pos % c.page_size * c.v.slot;
        }
    }
    const int64_t turn = min(max(pos, (int64_t)0), (int64_t)a.n_pos - 1) * (a.rot / 2);
    const float* cs = a.cos + turn;
    const float* sn = a.sin + turn;
    const T* k = static_cast<const T*>(a.k) + t * a.k_tok;
    const T* v = static_cast<const T*>(a.v) + t * a.v_tok;
    const T* q = static_cast<const T*>(a.q) + t * a.q_tok;
    T* kc = static_cast<T*>(c.k.p) + k_at;
    T* vc = static_cast<T*>(c.v.p) + v_at;
    T* qo = static_cast<T*>(a.q_out) + t * a.Hq * c.d;

    // items of a head that turns: pairs of vectors (half layout) or vectors of pairs, then those that are copied
    const int half = a.rot / 2, turned = a.interleaved ? (V == 1 ? half : a.rot / V) : half / V;
    const int per_turned = turned + (c.d - a.rot) / V, per_copied = c.d / V;
    const int heads = c.Hk + (a.q ? a.Hq : 0), items = heads * per_turned + c.Hk * per_copied;
    for (int e = tid; e < items; e += blockDim.x) {
        if (e >= heads * per_turned) {                     // a value
            const int i = e - heads * per_turned, h = i / per_copied, at = i % per_copied * V;
            if (k_at < 0) continue;
            Vec x;
            x.load(v + h * a.v_head + at);
            x.store(vc + h * c.v.head + at);
            continue;
        }
        const int h = e / per_turned, i = e % per_turned;
        const bool key = h < c.Hk;
        const T* src = key ? k + h * a.k_head : q + (h - c.Hk) * a.q_head;
        T* dst = key ? kc + h * c.k.head : qo + (int64_t)(h - c.Hk) * c.d;
        if (key && k_at < 0) continue;
        if (i >= turned) {
            const int at = a.rot + (i - turned) * V;
            Vec x;
            x.load(src + at);
            x.store(dst + at);
        } else if (!a.interleaved) {
            Vec x, y;
            x.load(src + i * V);
            y.load(src + half + i * V);
#pragma unroll
            for (int u = 0; u < V; ++u) {
                const float cc = cs[i * V + u], ss = sn[i * V + u], p = x.get(u), r = y.get(u);
                x.set(u, p * cc - r * ss);
                y.set(u, r * cc + p * ss);
            }
            x.store(dst + i * V);
            y.store(dst + half + i * V);
        } else if constexpr (V > 1) {
            Vec x;
            x.load(src + i * V);
#pragma unroll
            for (int u = 0; u < V; u += 2) {
                const float cc = cs[(i * V + u) / 2], ss = sn[(i * V + u) / 2], p = x.get(u), r = x.get(u + 1);
                x.set(u, p * cc - r * ss);
                x.set(u + 1, r * cc + p * ss);
            }
            x.store(dst + i * V);
        } else {
            const float cc = cs[i], ss = sn[i], p = mix::ld(src + 2 * i), r = mix::ld(src + 2 * i + 1);
            mix::st(dst + 2 * i, p * cc - r * ss);
            mix::st(dst + 2 * i + 1, r * cc + p * ss);
        }
    }
}

template <typename T>
cudaError_t typed(const PagedAppendArgs& a, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const PagedCache& c = a.c;
    auto fits = [](const void* p, int64_t x, int64_t y, int64_t z) {
        return (uintptr_t)p % 16 == 0 && x % V == 0 && y % V == 0 && z % V == 0;
    };
    const bool vec = c.d % V == 0 && a.rot % V == 0 && (a.interleaved || a.rot / 2 % V == 0) &&
                     fits(a.k, a.k_tok, a.k_head, 0) && fits(a.v, a.v_tok, a.v_head, 0) &&
                     (!a.q || (fits(a.q, a.q_tok, a.q_head, 0) && fits(a.q_out, 0, 0, 0))) &&
                     fits(c.k.p, c.k.page, c.k.slot, c.k.head) && fits(c.v.p, c.v.page, c.v.slot, c.v.head);
    const int64_t items = (int64_t)(2 * c.Hk + (a.q ? a.Hq : 0)) * c.d / (vec ? V : 1);
    const int threads = items > 192 ? 256 : items > 96 ? 128 : items > 48 ? 64 : 32;
    if (vec) paged_append_kernel<T, V><<<(unsigned)a.n_tokens, threads, 0, s>>>(a);
    else paged_append_kernel<T, 1><<<(unsigned)a.n_tokens, threads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t s) {
    if (a.n_tokens == 0) return cudaSuccess;
    return a.c.bf16 ? typed<bf16>(a, s) : typed<float>(a, s);
}

}  // namespace gdn
