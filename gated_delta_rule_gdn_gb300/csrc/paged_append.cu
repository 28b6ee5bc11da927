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

// The sequence of token t, the last n with cu[n] <= t, 32 candidates at a time (all lanes of a warp call it), with its offsets and
// its length, which are read beside the last candidates.
struct Place { int n, first, end, length; };
__device__ __forceinline__ Place place_of(const int32_t* cu, const int32_t* lengths, int N, int64_t t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = N;
    while (n > 32) {
        const int step = (n + 31) / 32, at = lane * step;
        const unsigned below = __ballot_sync(0xffffffffu, at < n && (at == 0 || cu[lo + at] <= t));
        const int hit = 31 - __clz(below);
        lo += hit * step;
        n = min(step, n - hit * step);
    }
    const int at = lo + min(lane, n - 1);
    const int first = cu[at], end = cu[at + 1], length = lengths[at];
    const int hit = 31 - __clz(__ballot_sync(0xffffffffu, lane < n && (lane == 0 || first <= t)));
    return {lo + hit, __shfl_sync(0xffffffffu, first, hit), __shfl_sync(0xffffffffu, end, hit), __shfl_sync(0xffffffffu, length, hit)};
}

template <typename T, int V>
__global__ void __launch_bounds__(256, 4) paged_append_kernel(const PagedAppendArgs a) {
    using Vec = mix::Vec<T, V>;
    const PagedCache& c = a.c;
    const int64_t t = blockIdx.x;
    const T* k = static_cast<const T*>(a.k) + t * a.k_tok;
    const T* v = static_cast<const T*>(a.v) + t * a.v_tok;
    const T* q = static_cast<const T*>(a.q) + t * a.q_tok;
    T* qo = static_cast<T*>(a.q_out) + t * a.Hq * c.d;

    // items of a head that turns: two vectors that turn with one another (half layout) or one of pairs, then those that are
    // copied; then the items of the values
    const int half = a.rot / 2, turned = a.interleaved ? (V == 1 ? half : a.rot / V) : half / V;
    const int per_turned = turned + (c.d - a.rot) / V, per_copied = c.d / V;
    const int heads = c.Hk + (a.q ? a.Hq : 0), all_turned = heads * per_turned, items = all_turned + c.Hk * per_copied;
    struct Item {
        Vec x, y;
        int h, at;                                         // head (keys, queries, then values), channel
        int pair;                                          // the index of its first angle, or -1
    };
    auto read = [&](int e, Item& it) {
        if (e >= items) {
            it.h = -1;
            return;
        }
        const T* src;
        if (e >= all_turned) {
            const int i = e - all_turned;
            it.h = heads + i / per_copied;
            it.at = i % per_copied * V;
            it.pair = -1;
            src = v + (it.h - heads) * a.v_head;
        } else {
            const int i = e % per_turned;
            it.h = e / per_turned;
            src = it.h < c.Hk ? k + it.h * a.k_head : q + (it.h - c.Hk) * a.q_head;
            it.pair = i >= turned ? -1 : a.interleaved ? (V == 1 ? i : i * V / 2) : i * V;
            it.at = i >= turned ? a.rot + (i - turned) * V : a.interleaved ? 2 * it.pair : it.pair;
        }
        it.x.load(src + it.at);
        if (it.pair >= 0) {
            if (!a.interleaved) it.y.load(src + half + it.at);
            else if (V == 1) it.y.load(src + it.at + 1);
        }
    };
    constexpr int AT_ONCE = 3;                             // items of a thread on their way while the slot is looked up
    Item it[AT_ONCE];
    const int tid = threadIdx.x;
#pragma unroll
    for (int u = 0; u < AT_ONCE; ++u) read(tid + u * blockDim.x, it[u]);

    int n = (int)t;
    int64_t pos;
    if (a.cu) {
        const Place at = place_of(a.cu, c.lengths, c.N, t);
        if (t < at.first || t >= at.end) return;           // a row behind the last sequence
        n = at.n;
        pos = at.length - (at.end - t);
    } else {
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
    const int64_t turn = min(max(pos, (int64_t)0), (int64_t)a.n_pos - 1) * half;
    const float* cs = a.cos + turn;
    const float* sn = a.sin + turn;
    auto write = [&](Item& i) {
        if (i.h < 0 || (k_at < 0 && (i.h < c.Hk || i.h >= heads))) return;
        T* dst = i.h >= heads ? static_cast<T*>(c.v.p) + v_at + (i.h - heads) * c.v.head
                 : i.h < c.Hk ? static_cast<T*>(c.k.p) + k_at + i.h * c.k.head
                              : qo + (int64_t)(i.h - c.Hk) * c.d;
        if (i.pair >= 0 && (!a.interleaved || V == 1)) {
#pragma unroll
            for (int u = 0; u < V; ++u) {
                const float cc = cs[i.pair + u], ss = sn[i.pair + u], p = i.x.get(u), r = i.y.get(u);
                i.x.set(u, p * cc - r * ss);
                i.y.set(u, r * cc + p * ss);
            }
            i.y.store(dst + (a.interleaved ? i.at + 1 : half + i.at));
        } else if constexpr (V > 1) {
            if (i.pair >= 0)
#pragma unroll
                for (int u = 0; u < V; u += 2) {
                    const float cc = cs[i.pair + u / 2], ss = sn[i.pair + u / 2], p = i.x.get(u), r = i.x.get(u + 1);
                    i.x.set(u, p * cc - r * ss);
                    i.x.set(u + 1, r * cc + p * ss);
                }
        }
        i.x.store(dst + i.at);
    };
    for (int e = tid; e < items; e += AT_ONCE * blockDim.x) {
        if (e != tid)
#pragma unroll
            for (int u = 0; u < AT_ONCE; ++u) read(e + u * blockDim.x, it[u]);
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) write(it[u]);
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
