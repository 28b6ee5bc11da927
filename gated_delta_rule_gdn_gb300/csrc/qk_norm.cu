// Norm of every query and key head with the position rotation in the same pass, and its gradients.
//   y = w x r,  r = 1 / sqrt(c sum x^2 + eps)  (c = 1/d: root mean square; c = 1: unit length)
//   the first `rot` channels of y turn by the angles of the token's position: pairs (i, i + rot/2), or (2i, 2i + 1)
//   interleaved.
// Backward: dy = the output's gradient turned back, dw = sum dy x r, e = w dy, dx = r (e - c r^2 x sum(x e)).
// Bound by HBM: every head is read once and written once (backward: read with its gradient, written once).  Measured: 16,384
// tokens x 32 heads of 128 in bf16 without rotation 43.7 us forward (268 MB, 90 % of the copy rate) and 68 us backward (403 MB,
// 88 %); 16,384 tokens x 40 heads, half of each rotated, 65 us forward (336 MB, 76 %) and 107 us backward (503 MB, 69 %), where
// the shuffles and the angles' latency show, in fp32 127 (78 %) and 167 us (89 %).
//
// Vector kernels: G neighbouring lanes hold a head, E = 8 or 4 channels each, and a group of lanes takes N heads of one token,
// so that the token's angles are read once for them.  Blocks are persistent; each thread's inputs of the next shares come
// through kSlots slots of its own in shared memory, so that loads are under way all the time.  The rotation's
// partner is in the same lane (interleaved), or in the lane rot / 2E away.  Heads whose size, rotation or alignment
// does not go in steps of 4 channels take the scalar kernels, a warp per head.

#include <type_traits>

#include "mixer.h"
#include "mixer_common.cuh"

namespace gdn {
namespace {

using mix::bf16;
using mix::ld;
using mix::st;

constexpr int kMaxD = 256, kThreads = 256;

__device__ __forceinline__ int position(const QkNormArgs& a, int64_t tok) {
    const int p = a.pos ? a.pos[tok] : (int)((unsigned)tok % (unsigned)a.T);    // (tokens times heads fit 31 bits)
    return min(max(p, 0), a.n_pos - 1);
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int m = G / 2; m > 0; m >>= 1) v += __shfl_xor_sync(~0u, v, m, G);
    return v;
}

// E channels in accesses of at most 16 bytes
template <typename T, int E>
struct Chunk {
    static constexpr int N = sizeof(T) * E > 16 ? 16 / sizeof(T) : E, kParts = E / N;
    using Part = mix::Vec<T, N>;
    Part v[kParts];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < E / N; ++i) v[i].load(p + i * N);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < E / N; ++i) v[i].zero();
    }
    __device__ __forceinline__ float get(int i) const { return v[i / N].get(i % N); }
    __device__ __forceinline__ void set(int i, float x) { v[i / N].set(i % N, x); }
    __device__ __forceinline__ void store(T* p) const {
#pragma unroll
        for (int i = 0; i < E / N; ++i) v[i].store(p + i * N);
    }
};

enum Rotation { kNone, kHalves, kInterleaved };

// The angles of a lane's channels at position p, for turning them forward (sign = 1) or back (sign = -1); for halves `sin` has the
// sign that the forward rotation gives the partner's term.  A lane past the rotated channels keeps its own: for halves it is its own
// partner, with y / 2 + y / 2, interleaved it selects.  (By cos = 1 and sin = 0 an infinity would make its neighbour NaN.  Against
// that form a branch around the turn took 3 to 18 % longer forward, this 1 % or less and, interleaved, 2 %.)
template <int E, int ROT>
struct Angles {
    float c[ROT == kInterleaved ? E / 2 : E], s[ROT == kInterleaved ? E / 2 : E];
    int partner;
    bool in;
    __device__ __forceinline__ void load(const QkNormArgs& a, int p, int lane, float sign) {
        const int j = lane * E, half = a.rot / 2;
        constexpr int N = ROT == kInterleaved ? E / 2 : E;
        in = j < a.rot;
        const bool low = j < half;
        const int at = ROT == kInterleaved ? j / 2 : (low ? j : j - half);
        partner = in ? (low ? lane + half / E : lane - half / E) : lane;
        const float* cp = a.cos + (int64_t)p * half + at;
        const float* sp = a.sin + (int64_t)p * half + at;
        Chunk<float, N> x, y;
        if (in) x.load(cp);
        if (in) y.load(sp);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            c[i] = in ? x.get(i) : 0.5f;
            s[i] = in ? y.get(i) : sign * 0.5f;
        }
        if (ROT == kHalves && low)
#pragma unroll
            for (int i = 0; i < N; ++i) s[i] = -s[i];
    }
    template <int G>
    __device__ __forceinline__ void turn(float (&y)[E], float sign) const {
        if (ROT == kHalves) {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float o = __shfl_sync(~0u, y[i], partner, G);
                y[i] = fmaf(sign * s[i], o, y[i] * c[i]);
            }
        } else if (ROT == kInterleaved) {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                const float u = y[2 * i], v = y[2 * i + 1];
                const float t = fmaf(u, c[i], -sign * s[i] * v), w = fmaf(v, c[i], sign * s[i] * u);
                y[2 * i] = in ? t : u;
                y[2 * i + 1] = in ? w : v;
            }
        }
    }
};

// A group's share of the work: up to N heads of q, or of k, of one token.  The token's shares are those of q, then of k.
struct Shares { unsigned of_q, all; };
template <typename T, int E, int G, int N>
struct Share {
    unsigned tok;
    int which, count, j0;             // tensor, heads, the lane's first channel
    const T* x;                       // the lane's channels of the first head in the input, and the same in contiguous
    size_t at;                        // tensors
    int64_t step;                     // between the input's heads
    // (a share past the last has no heads)
    __device__ __forceinline__ Share(const QkNormArgs& a, const Shares& sh, unsigned item, unsigned items) {
        const bool real = item < items;
        if (!real) item = items - 1;
        tok = item / sh.all;
        unsigned part = item - tok * sh.all;
        which = part >= sh.of_q;
        if (which) part -= sh.of_q;
        const int h = (int)part * N, H = which ? a.H[1] : a.H[0];
        j0 = (int)(threadIdx.x % G) * E;
        count = real && j0 < a.d ? min(H - h, N) : 0;
        step = which ? a.head_stride[1] : a.head_stride[0];
        x = static_cast<const T*>(which ? a.in[1] : a.in[0]) + (int64_t)tok * (which ? a.tok_stride[1] : a.tok_stride[0]) +
            h * step + j0;
        at = ((size_t)tok * H + h) * a.d + j0;
    }
};
template <typename T, int E>
__device__ __forceinline__ void copy_chunk(Chunk<T, E>* dst, int pitch, const T* src, bool in, const void* any) {
#pragma unroll
    for (int i = 0; i < Chunk<T, E>::kParts; ++i)
        mix::copy_async(reinterpret_cast<typename Chunk<T, E>::Part*>(dst) + i * pitch,
                        in ? src + i * Chunk<T, E>::N : static_cast<const T*>(any), in);
}
template <typename T, int E>
__device__ __forceinline__ Chunk<T, E> read_chunk(const Chunk<T, E>* src, int pitch) {
    Chunk<T, E> c;
#pragma unroll
    for (int i = 0; i < Chunk<T, E>::kParts; ++i) c.v[i] = reinterpret_cast<const typename Chunk<T, E>::Part*>(src)[i * pitch];
    return c;
}

// Without rotation there is little to wait for but the heads: a block for every share is then faster than persistent ones
// (16,384 tokens x 32 heads of 128: 43 and 52 us); with it the angles' latency is worth hiding (16,384 tokens x 40 heads: 78 us
// with a block for every share, 68 us so).
template <int ROT> constexpr int kSlots = ROT == kNone ? 1 : 2;
constexpr int kBwdSlots = 2;

template <typename T, int E, int G, int ROT, int N>
__global__ void __launch_bounds__(kThreads) qk_fwd_kernel(const QkNormArgs a, const Shares sh, const unsigned items) {
    using C = Chunk<T, E>;
    constexpr unsigned kGroups = kThreads / G;
    extern __shared__ __align__(16) unsigned char s_raw[];
    auto* buf = reinterpret_cast<typename C::Part*>(s_raw) + threadIdx.x;     // [slots][N][parts][256]
    const auto slot = [&](int k, int i) { return reinterpret_cast<C*>(buf + ((k * N + i) * C::kParts) * kThreads); };
    const unsigned stride = gridDim.x * kGroups, first = blockIdx.x * kGroups + threadIdx.x / G;
    const auto fetch = [&](unsigned item, int k) {
        const Share<T, E, G, N> w(a, sh, item, items);
#pragma unroll
        for (int i = 0; i < N; ++i) copy_chunk<T, E>(slot(k, i), kThreads, w.x + i * w.step, i < w.count, a.in[0]);
        mix::copies_close();
    };
#pragma unroll
    for (int k = 0; k < kSlots<ROT>; ++k) fetch(first + k * stride, k);
    int k = 0;
    // (all groups of a block go round as often as its first)
    for (unsigned item = first, base = blockIdx.x * kGroups; base < items; item += stride, base += stride) {
        const Share<T, E, G, N> w(a, sh, item, items);
        Angles<E, ROT> ang;
        if (ROT != kNone) ang.load(a, position(a, w.tok), (int)threadIdx.x % G, 1.f);
        const float* wt = w.which ? a.w[1] : a.w[0];
        float weight[E];
#pragma unroll
        for (int e = 0; e < E; ++e) weight[e] = wt && w.count > 0 ? wt[w.j0 + e] : 1.f;
        T* y = static_cast<T*>(w.which ? a.out[1] : a.out[0]) + w.at;
        mix::copies_wait<kSlots<ROT> - 1>();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            C x = read_chunk<T, E>(slot(k, i), kThreads);
            float v[E], ss = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                v[e] = x.get(e);
                ss = fmaf(v[e], v[e], ss);
            }
            const float r = rsqrtf(fmaf(a.c, group_sum<G>(ss), a.eps));
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] *= r * weight[e];
            ang.template turn<G>(v, 1.f);
#pragma unroll
            for (int e = 0; e < E; ++e) x.set(e, v[e]);
            if (i < w.count) x.store(y);
            y += a.d;
        }
        fetch(item + kSlots<ROT> * stride, k);
        k = k + 1 == kSlots<ROT> ? 0 : k + 1;
    }
}

// The weight gradients of a block's heads stay in registers and leave as one row of partial sums.
template <typename T, int E, int G, int ROT, int N>
__global__ void __launch_bounds__(kThreads, 2) qk_bwd_kernel(const QkNormArgs a, const Shares sh, const unsigned items,
                                                             float* part) {
    using C = Chunk<T, E>;
    constexpr unsigned kGroups = kThreads / G;
    mix::let_next();
    extern __shared__ __align__(16) unsigned char s_raw[];
    auto* buf = reinterpret_cast<typename C::Part*>(s_raw) + threadIdx.x;     // [kBwdSlots][N][x, dz][parts][256]
    const auto slot = [&](int k, int i, int z) {
        return reinterpret_cast<C*>(buf + (((k * N + i) * 2 + z) * C::kParts) * kThreads);
    };
    const unsigned stride = gridDim.x * kGroups, first = blockIdx.x * kGroups + threadIdx.x / G;
    const auto fetch = [&](unsigned item, int k) {
        const Share<T, E, G, N> w(a, sh, item, items);
        const T* dp = static_cast<const T*>(w.which ? a.dout[1] : a.dout[0]) + w.at;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            copy_chunk<T, E>(slot(k, i, 0), kThreads, w.x + i * w.step, i < w.count, a.in[0]);
            copy_chunk<T, E>(slot(k, i, 1), kThreads, dp + (size_t)i * a.d, i < w.count, a.in[0]);
        }
        mix::copies_close();
    };
#pragma unroll
    for (int k = 0; k < kBwdSlots; ++k) fetch(first + k * stride, k);
    float acc[2][E] = {};
    int k = 0;
    for (unsigned item = first, base = blockIdx.x * kGroups; base < items; item += stride, base += stride) {
        const Share<T, E, G, N> w(a, sh, item, items);
        Angles<E, ROT> ang;
        if (ROT != kNone) ang.load(a, position(a, w.tok), (int)threadIdx.x % G, -1.f);
        const float* wt = w.which ? a.w[1] : a.w[0];
        float weight[E], sum[E] = {};
#pragma unroll
        for (int e = 0; e < E; ++e) weight[e] = wt && w.count > 0 ? wt[w.j0 + e] : 1.f;
        T* out = static_cast<T*>(w.which ? a.out[1] : a.out[0]) + w.at;
        mix::copies_wait<kBwdSlots - 1>();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            C x = read_chunk<T, E>(slot(k, i, 0), kThreads);
            const C dz = read_chunk<T, E>(slot(k, i, 1), kThreads);
            float e[E], v[E], ss = 0.f, xe = 0.f;
#pragma unroll
            for (int c = 0; c < E; ++c) {
                e[c] = dz.get(c);
                v[c] = x.get(c);
                ss = fmaf(v[c], v[c], ss);
            }
            ang.template turn<G>(e, -1.f);
            const float r = rsqrtf(fmaf(a.c, group_sum<G>(ss), a.eps));
#pragma unroll
            for (int c = 0; c < E; ++c) {
                v[c] *= r;
                sum[c] = fmaf(e[c], v[c], sum[c]);
                e[c] *= weight[c];
                xe = fmaf(v[c], e[c], xe);
            }
            xe = group_sum<G>(xe) * a.c;
#pragma unroll
            for (int c = 0; c < E; ++c) x.set(c, r * fmaf(-v[c], xe, e[c]));
            if (i < w.count) x.store(out);
            out += a.d;
        }
        fetch(item + kBwdSlots * stride, k);
        k = k + 1 == kBwdSlots ? 0 : k + 1;
        // (heads that a share does not have were copied as zeros and add nothing)
#pragma unroll
        for (int c = 0; c < E; ++c) {
            acc[0][c] += w.which ? 0.f : sum[c];
            acc[1][c] += w.which ? sum[c] : 0.f;
        }
    }
    if (!part) return;
    mix::copies_wait<0>();
    __syncthreads();
    auto& sw = *reinterpret_cast<float(*)[2][kGroups][G * E]>(s_raw);         // (the slots are done with)
    const int g = threadIdx.x / G, lane = threadIdx.x % G;
#pragma unroll
    for (int c = 0; c < E; ++c) {
        sw[0][g][lane * E + c] = acc[0][c];
        sw[1][g][lane * E + c] = acc[1][c];
    }
    __syncthreads();
    for (int j = threadIdx.x; j < 2 * a.d; j += kThreads) {
        float s = 0.f;
        for (unsigned i = 0; i < kGroups; ++i) s += sw[j / a.d][i][j % a.d];
        part[(size_t)blockIdx.x * 2 * a.d + j] = s;
    }
}

// ---------------------------------------------------------------------------- any size and alignment: a warp per head

constexpr int kWarps = kThreads / 32;

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

template <typename T>
__global__ void __launch_bounds__(kThreads) qk_fwd_any_kernel(const QkNormArgs a) {
    __shared__ float buf[kWarps][kMaxD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t id = (int64_t)blockIdx.x * kWarps + warp;
    const int heads = a.H[0] + a.H[1];
    const int64_t tok = (unsigned)id / (unsigned)heads;
    const int hh = (int)((unsigned)id % (unsigned)heads), which = hh >= a.H[0], h = which ? hh - a.H[0] : hh;
    if (tok >= a.n) return;
    const T* x = static_cast<const T*>(a.in[which]) + tok * a.tok_stride[which] + h * a.head_stride[which];
    T* y = static_cast<T*>(a.out[which]) + (tok * a.H[which] + h) * a.d;
    float v[kMaxD / 32], ss = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxD / 32; ++i) {
        const int j = lane + 32 * i;
        v[i] = j < a.d ? ld(x + j) : 0.f;
        ss = fmaf(v[i], v[i], ss);
    }
    const float r = rsqrtf(fmaf(a.c, group_sum<32>(ss), a.eps));
#pragma unroll
    for (int i = 0; i < kMaxD / 32; ++i) {
        const int j = lane + 32 * i;
        if (j < a.d) buf[warp][j] = v[i] * r * (a.w[which] ? a.w[which][j] : 1.f);
    }
    __syncwarp();
    const int p = a.rot ? position(a, tok) : 0;
#pragma unroll
    for (int i = 0; i < kMaxD / 32; ++i) {
        const int j = lane + 32 * i;
        if (j >= a.d) break;
        float u = buf[warp][j];
        if (j < a.rot) {
            int o, k;
            float sg;
            pair_of(a, j, &o, &sg, &k);
            const int64_t at = (int64_t)p * (a.rot >> 1) + k;
            u = u * a.cos[at] + sg * buf[warp][o] * a.sin[at];
        }
        st(y + j, u);
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 3) qk_bwd_any_kernel(const QkNormArgs a, float* part) {
    __shared__ float buf[kWarps][kMaxD];
    __shared__ float dw[2][kWarps][kMaxD];
    mix::let_next();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int heads = a.H[0] + a.H[1];
    float acc[2][kMaxD / 32] = {};
    for (int64_t id = (int64_t)blockIdx.x * kWarps + warp; id < a.n * heads; id += (int64_t)gridDim.x * kWarps) {
        const int64_t tok = (unsigned)id / (unsigned)heads;
        const int hh = (int)((unsigned)id % (unsigned)heads), which = hh >= a.H[0], h = which ? hh - a.H[0] : hh;
        const T* x = static_cast<const T*>(a.in[which]) + tok * a.tok_stride[which] + h * a.head_stride[which];
        const T* dz = static_cast<const T*>(a.dout[which]) + (tok * a.H[which] + h) * a.d;
        T* dx = static_cast<T*>(a.out[which]) + (tok * a.H[which] + h) * a.d;
        float ss = 0.f, xe = 0.f, e[kMaxD / 32], xv[kMaxD / 32];       // (all loads first)
#pragma unroll
        for (int i = 0; i < kMaxD / 32; ++i) {
            const int j = lane + 32 * i;
            e[i] = j < a.d ? ld(dz + j) : 0.f;
            xv[i] = j < a.d ? ld(x + j) : 0.f;
        }
        if (a.rot > 0) {
            const int p = position(a, tok);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kMaxD / 32; ++i) buf[warp][lane + 32 * i] = e[i];
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kMaxD / 32; ++i) {
                const int j = lane + 32 * i;
                if (j >= a.rot) continue;
                int o, k;
                float sg;
                pair_of(a, j, &o, &sg, &k);
                const int64_t at = (int64_t)p * (a.rot >> 1) + k;
                e[i] = e[i] * a.cos[at] - sg * buf[warp][o] * a.sin[at];
            }
        }
#pragma unroll
        for (int i = 0; i < kMaxD / 32; ++i) ss = fmaf(xv[i], xv[i], ss);
        const float r = rsqrtf(fmaf(a.c, group_sum<32>(ss), a.eps));
#pragma unroll
        for (int i = 0; i < kMaxD / 32; ++i) {
            const int j = lane + 32 * i;
            if (j >= a.d) continue;
            const float t = e[i] * xv[i] * r;
            if (which) acc[1][i] += t; else acc[0][i] += t;
            if (a.w[which]) e[i] *= a.w[which][j];
            xe = fmaf(xv[i], e[i], xe);
        }
        xe = group_sum<32>(xe) * a.c * r * r;
#pragma unroll
        for (int i = 0; i < kMaxD / 32; ++i) {
            const int j = lane + 32 * i;
            if (j < a.d) st(dx + j, r * (e[i] - xv[i] * xe));
        }
    }
    if (!part) return;
#pragma unroll
    for (int i = 0; i < kMaxD / 32; ++i) {
        dw[0][warp][lane + 32 * i] = acc[0][i];
        dw[1][warp][lane + 32 * i] = acc[1][i];
    }
    __syncthreads();
    for (int j = threadIdx.x; j < 2 * a.d; j += kThreads) {
        float s = 0.f;
        for (int i = 0; i < kWarps; ++i) s += dw[j / a.d][i][j % a.d];
        part[(size_t)blockIdx.x * 2 * a.d + j] = s;
    }
}

// column sums of part [rows][2 d]: 8 columns a block, 32 row lanes, joined in order
__global__ void __launch_bounds__(256) qk_dw_kernel(const float* part, int rows, int d, float* dwq, float* dwk) {
    __shared__ float s[32][9];
    const int c = threadIdx.x % 8, w = threadIdx.x / 8, j = blockIdx.x * 8 + c;
    mix::wait_behind();
    float acc = 0.f;
    if (j < 2 * d)
#pragma unroll 4
        for (int r = w; r < rows; r += 32) acc += part[(size_t)r * 2 * d + j];
    s[w][c] = acc;
    __syncthreads();
    if (w == 0 && j < 2 * d) {
        float t = 0.f;
        for (int i = 0; i < 32; ++i) t += s[i][c];
        float* out = j < d ? dwq : dwk;
        if (out) out[j < d ? j : j - d] = t;
    }
}

// The channels a lane takes in the vector kernels: 8 or 4, whichever everything goes in steps of, or 0 if neither (twice 16,384
// tokens x 32 heads of 128 in bf16: forward 78 us, 103, and 250 with the scalar kernel; backward 109, 134 and 400).
int channels_a_lane(const QkNormArgs& a, bool backward) {
    for (int E = 8; E >= 4; E /= 2) {
        const size_t size = (a.bf16 ? 2 : 4) * E, bytes = size < 16 ? size : 16;
        const size_t table = a.interleaved ? 2 * E : (E < 4 ? E : 4) * 4;
        const auto al = [](const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
        bool ok = a.d % E == 0 && a.d <= 32 * E;
        if (a.rot > 0)
            ok = ok && (a.interleaved ? a.rot % E == 0 : a.rot % (2 * E) == 0) && al(a.cos, table < 16 ? table : 16) &&
                 al(a.sin, table < 16 ? table : 16);
        for (int i = 0; i < 2; ++i)
            ok = ok && a.tok_stride[i] % E == 0 && a.head_stride[i] % E == 0 && al(a.in[i], bytes) && al(a.out[i], bytes) &&
                 (!backward || al(a.dout[i], bytes));
        if (ok) return E;
    }
    return 0;
}

constexpr unsigned kFwdBlocks = 152 * 4, kBwdBlocks = 152 * 2, kAnyBlocks = 152 * 3;
Shares shares_of(const QkNormArgs& a, int N) {
    const unsigned q = (a.H[0] + N - 1) / N, k = (a.H[1] + N - 1) / N;
    return {q, q + k};
}
cudaError_t allow_smem(const void* kernel, size_t bytes) {
    return bytes > 48 * 1024 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes)
                             : cudaSuccess;
}
constexpr int kFwdHeads = 4;
template <typename T> constexpr int kBwdHeads = sizeof(T) == 2 ? 4 : 2;       // (two inputs, 64 KB of slots a block)
// Heads a share: as above, or one where neither tensor has as many as half of that.
template <int N, typename F>
void by_heads(const QkNormArgs& a, F f) {
    if (2 * a.H[0] <= N && 2 * a.H[1] <= N) f(std::integral_constant<int, 1>{});
    else f(std::integral_constant<int, N>{});
}

// f(channels a lane, group size, rotation) as compile-time constants
template <typename F>
void by_shape(const QkNormArgs& a, int E, F f) {
    const auto rot = [&](auto e, auto g) {
        if (a.rot == 0) f(e, g, std::integral_constant<int, kNone>{});
        else if (a.interleaved) f(e, g, std::integral_constant<int, kInterleaved>{});
        else f(e, g, std::integral_constant<int, kHalves>{});
    };
    using std::integral_constant;
    if (E == 4) {
        if (a.d <= 64) rot(integral_constant<int, 4>{}, integral_constant<int, 16>{});
        else rot(integral_constant<int, 4>{}, integral_constant<int, 32>{});
    } else if (a.d <= 64) rot(integral_constant<int, 8>{}, integral_constant<int, 8>{});
    else if (a.d <= 128) rot(integral_constant<int, 8>{}, integral_constant<int, 16>{});
    else rot(integral_constant<int, 8>{}, integral_constant<int, 32>{});
}

template <typename T>
cudaError_t fwd(const QkNormArgs& a, cudaStream_t s) {
    if (const int E = channels_a_lane(a, false)) {
        cudaError_t err = cudaSuccess;
        by_heads<kFwdHeads>(a, [&](auto heads) {
            const Shares sh = shares_of(a, heads.value);
            const unsigned items = (unsigned)(a.n * sh.all);     // (at most tokens times heads, which fits)
            by_shape(a, E, [&](auto e, auto g, auto rot) {
                const unsigned per = kThreads / g.value, want = (items + per - 1) / per;
                const auto kernel = qk_fwd_kernel<T, e.value, g.value, rot.value, heads.value>;
                const size_t smem = (size_t)kSlots<rot.value> * heads.value * kThreads * e.value * sizeof(T);
                err = allow_smem(reinterpret_cast<const void*>(kernel), smem);
                if (err == cudaSuccess)
                    kernel<<<rot.value == kNone || want < kFwdBlocks ? want : kFwdBlocks, kThreads, smem, s>>>(a, sh, items);
            });
        });
        if (err != cudaSuccess) return err;
    } else {
        const int64_t rows = a.n * (a.H[0] + a.H[1]);
        qk_fwd_any_kernel<T><<<(unsigned)((rows + kWarps - 1) / kWarps), kThreads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t bwd(const QkNormArgs& a, cudaStream_t s) {
    const bool weights = a.dw[0] || a.dw[1];
    float* part = weights ? static_cast<float*>(a.ws) : nullptr;
    int blocks = 0;                            // none without tokens: the weight gradients are then zero
    const int E = a.n > 0 ? channels_a_lane(a, true) : 0;
    if (E > 0) {
        cudaError_t err = cudaSuccess;
        by_heads<kBwdHeads<T>>(a, [&](auto heads) {
            const Shares sh = shares_of(a, heads.value);
            const unsigned items = (unsigned)(a.n * sh.all);
            by_shape(a, E, [&](auto e, auto g, auto rot) {
                const unsigned per = kThreads / g.value, want = (items + per - 1) / per;
                blocks = (int)(want < kBwdBlocks ? want : kBwdBlocks);
                const auto kernel = qk_bwd_kernel<T, e.value, g.value, rot.value, heads.value>;
                const size_t slots = 2 * (size_t)kBwdSlots * heads.value * kThreads * e.value * sizeof(T);
                const size_t sums = 2 * (size_t)kThreads * e.value * sizeof(float), smem = slots > sums ? slots : sums;
                err = allow_smem(reinterpret_cast<const void*>(kernel), smem);
                if (err == cudaSuccess) kernel<<<blocks, kThreads, smem, s>>>(a, sh, items, part);
            });
        });
        if (err != cudaSuccess) return err;
    } else if (a.n > 0) {
        const int64_t want = (a.n * (a.H[0] + a.H[1]) + kWarps - 1) / kWarps;
        blocks = (int)(want < (int64_t)kAnyBlocks ? want : (int64_t)kAnyBlocks);
        qk_bwd_any_kernel<T><<<blocks, kThreads, 0, s>>>(a, part);
    }
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess || !weights) return err;
    return mix::launch_behind(qk_dw_kernel, (2 * a.d + 7) / 8, 256, 0, blocks > 0, s, part, blocks, a.d, a.dw[0], a.dw[1]);
}

}  // namespace

size_t qk_norm_workspace_bytes(const QkNormArgs& a) {
    const int64_t want = (a.n * (a.H[0] + a.H[1]) + 7) / 8;          // at least the blocks of either kernel
    return (size_t)(want < (int64_t)kAnyBlocks ? want : (int64_t)kAnyBlocks) * 2 * a.d * sizeof(float);
}
cudaError_t launch_qk_norm_fwd(const QkNormArgs& a, cudaStream_t s) { return a.bf16 ? fwd<bf16>(a, s) : fwd<float>(a, s); }
cudaError_t launch_qk_norm_bwd(const QkNormArgs& a, cudaStream_t s) { return a.bf16 ? bwd<bf16>(a, s) : bwd<float>(a, s); }

}  // namespace gdn
