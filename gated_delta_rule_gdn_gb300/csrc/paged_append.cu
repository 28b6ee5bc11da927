// Appending keys and values to a paged cache, with the position rotation of keys (and queries) on the way.
//
// One block takes one new token.  A thread keeps one place in the head (two vectors of 16 bytes that turn with one another, one of
// interleaved pairs, or one that is copied) and its angles, and takes that place of every few heads; so the angles are read once
// for all of them.  Each value is read and written once, which is the bound where there are many tokens (16,384 tokens of 48 heads
// of 128: 80 us, 75 % of the copy rate, 12 small blocks an SM; 97 us in 6 of twice the threads, and 107 with the angles read for
// each head and divisions for each item, when instructions were the bound).  A decode step waits for the chain from the length over
// the table to the store.

#include "mixer_common.cuh"
#include "paged.h"

namespace gdn {
namespace {

using mix::bf16;

// The sequence of token t, the last n with cu[n] <= t, 32 candidates at a time (all lanes of a warp call it), with its offsets and
// its length, which are read beside the last candidates.
struct Place { int n, first, end, length; };
__device__ __forceinline__ Place place_of(const int32_t* cu, const int32_t* lengths, int N, int64_t t, int lane) {
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

// N angles' cosines or sines, 16 or 8 bytes an access where N allows (a place's angles begin on such a boundary).
template <int N>
__device__ __forceinline__ void angles(const float* p, float* d) {
    if constexpr (N == 4) {
        const float4 x = *reinterpret_cast<const float4*>(p);
        d[0] = x.x; d[1] = x.y; d[2] = x.z; d[3] = x.w;
    } else if constexpr (N == 2) {
        const float2 x = *reinterpret_cast<const float2*>(p);
        d[0] = x.x; d[1] = x.y;
    } else if constexpr (N == 1) {
        d[0] = *p;
    }
}

// blockDim.x threads for the places of a head, blockDim.y heads at a time.
template <typename T, int V>
__global__ void __launch_bounds__(128, 12) paged_append_kernel(const PagedAppendArgs a) {
    using Vec = mix::Vec<T, V>;
    const PagedCache& c = a.c;
    const int64_t t = blockIdx.x;
    const int tx = threadIdx.x, ty = threadIdx.y;
    int n = (int)t;
    int64_t pos;
    if (a.cu) {
        const Place at = place_of(a.cu, c.lengths, c.N, t, (ty * blockDim.x + tx) & 31);
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
    const int half = a.rot / 2;
    const int64_t turn = min(max(pos, (int64_t)0), (int64_t)a.n_pos - 1) * half;
    const T* k = static_cast<const T*>(a.k) + t * a.k_tok;
    const T* v = static_cast<const T*>(a.v) + t * a.v_tok;
    const T* q = static_cast<const T*>(a.q) + t * a.q_tok;
    T* kc = static_cast<T*>(c.k.p) + k_at;
    T* vc = static_cast<T*>(c.v.p) + v_at;
    T* qo = static_cast<T*>(a.q_out) + t * a.Hq * c.d;

    // places of a head that turns: two vectors (half layout, and single elements) or one of pairs, then those that are copied
    const bool pairs = a.interleaved && V > 1;
    const int turned = pairs ? a.rot / V : half / V, per_turned = turned + (c.d - a.rot) / V;
    const int keys = k_at < 0 ? c.Hk : 0, turning = c.Hk + (a.q ? a.Hq : 0);     // heads: keys (if there is a slot), queries
    for (int i = tx; i < per_turned; i += blockDim.x) {
        const bool turns = i < turned;
        const int at = !turns ? a.rot + (i - turned) * V : a.interleaved && V == 1 ? 2 * i : i * V;
        const int other = a.interleaved ? at + 1 : half + at;
        float cs[V], sn[V];
        if (turns) {
            const float* cp = a.cos + turn + (pairs ? at / 2 : i * V);
            const float* sp = a.sin + turn + (pairs ? at / 2 : i * V);
            angles<V / 2>(cp, cs);                         // (pairs have half as many angles as channels)
            angles<V / 2>(sp, sn);
            if (!pairs) {
                angles<V - V / 2>(cp + V / 2, cs + V / 2);
                angles<V - V / 2>(sp + V / 2, sn + V / 2);
            }
        }
#pragma unroll 1
        for (int h = keys + ty; h < turning; h += blockDim.y) {
            const bool key = h < c.Hk;
            const T* src = key ? k + h * a.k_head : q + (h - c.Hk) * a.q_head;
            T* dst = key ? kc + h * c.k.head : qo + (int64_t)(h - c.Hk) * c.d;
            Vec x, y;
            x.load(src + at);
            if (turns && !pairs) {
                y.load(src + other);
#pragma unroll
                for (int u = 0; u < V; ++u) {
                    const float p = x.get(u), r = y.get(u);
                    x.set(u, p * cs[u] - r * sn[u]);
                    y.set(u, r * cs[u] + p * sn[u]);
                }
                y.store(dst + other);
            } else if (turns) {
                if constexpr (V > 1)
#pragma unroll
                    for (int u = 0; u < V; u += 2) {
                        const float p = x.get(u), r = x.get(u + 1);
                        x.set(u, p * cs[u / 2] - r * sn[u / 2]);
                        x.set(u + 1, r * cs[u / 2] + p * sn[u / 2]);
                    }
            }
            x.store(dst + at);
        }
    }
    if (k_at < 0) return;
    for (int i = tx; i < c.d / V; i += blockDim.x)
#pragma unroll 1
        for (int h = ty; h < c.Hk; h += blockDim.y) {
            Vec x;
            x.load(v + h * a.v_head + i * V);
            x.store(vc + h * c.v.head + i * V);
        }
}

template <typename T>
cudaError_t typed(const PagedAppendArgs& a, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const PagedCache& c = a.c;
    auto fits = [](const void* p, int64_t x, int64_t y, int64_t z) {
        return (uintptr_t)p % 16 == 0 && x % V == 0 && y % V == 0 && z % V == 0;
    };
    const bool vec = c.d % V == 0 && a.rot % V == 0 && (a.interleaved || a.rot / 2 % V == 0) && fits(a.cos, 0, 0, 0) && fits(a.sin, 0, 0, 0) &&
                     fits(a.k, a.k_tok, a.k_head, 0) && fits(a.v, a.v_tok, a.v_head, 0) &&
                     (!a.q || (fits(a.q, a.q_tok, a.q_head, 0) && fits(a.q_out, 0, 0, 0))) &&
                     fits(c.k.p, c.k.page, c.k.slot, c.k.head) && fits(c.v.p, c.v.page, c.v.slot, c.v.head);
    const int heads = c.Hk + (a.q ? a.Hq : 0), places = (c.d - (vec && a.interleaved ? 0 : a.rot / 2)) / (vec ? V : 1);
    int x = 1, y = 128;                                    // as many threads a head as it has places, and no more heads than there are
    while (x < places && x < 32) x *= 2;
    y /= x;
    while (y / 2 >= heads && x * y > 32) y /= 2;
    if (vec) paged_append_kernel<T, V><<<(unsigned)a.n_tokens, dim3(x, y), 0, s>>>(a);
    else paged_append_kernel<T, 1><<<(unsigned)a.n_tokens, dim3(x, y), 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t s) {
    if (a.n_tokens == 0) return cudaSuccess;
    return a.c.bf16 ? typed<bf16>(a, s) : typed<float>(a, s);
}

}  // namespace gdn
