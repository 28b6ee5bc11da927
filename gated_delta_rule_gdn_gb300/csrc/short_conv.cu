// Short causal depthwise convolution with its activation, its gradients, and the decode step.
//   p_t = b + sum_j w_j x_{t - W + 1 + j},  y_t = silu(p_t) or p_t; inputs before a sequence's first token are its
//   initial state (its last W - 1 inputs, oldest first) or zero.
// Backward: ds = dy silu'(p), dx_t = sum_j w_j ds_{t + W - 1 - j}, dw_j = sum_t ds_t x_{t - W + 1 + j}, db = sum ds.
// Bound by HBM: x is read once and y written once (backward: x and dy read once, dx written once).  Measured in bf16, width 4
// with silu: 16,384 tokens x 6144 channels 69 us (403 MB, 86 % of the copy rate), in fp32 128 us (93 %) and 197 us backward (91 %);
// 65,536 packed tokens x 4096 channels 166 us forward (1.07 GB, 95 %) and 341 us backward (1.61 GB, 70 %; 29 instructions an element
// and 16 warps an SM show there).
//
// A thread walks a run of tokens of V neighbouring channels with the last W inputs in registers, a warp 32 V channels;
// the W - 1 tokens around a run that its neighbours walk too come out of L2.  The backward walks W - 1 tokens further, for
// the ds that its last tokens need, and keeps its sums of dw and db in registers; a block adds up its 8 runs and a second
// kernel the blocks, in order.  Rows of sequence states (the final state, the initial state's gradient) are formed by
// blocks of their own at the end of the grid.

#include <type_traits>

#include "mixer.h"
#include "mixer_common.cuh"

namespace gdn {
namespace {

using mix::bf16;
using mix::Vec;

// A thread's inputs come through a ring of its own in shared memory, kRing tokens deep, kChunk tokens a copy group: 16
// tokens forward; 8 backward, where two rings of 16 leave room for one block less in fp32 (52 and 70 us, B2 T4096 D2048).
constexpr int kWarps = 8, kChunk = 4, kFwdRing = 16, kBwdRing = 8, kThreads = kWarps * 32;
static_assert(kFwdRing % kChunk == 0 && kBwdRing % kChunk == 0, "whole groups");

__device__ __forceinline__ float ex2(float x) { float y; asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x)); return y; }
__device__ __forceinline__ float rcp(float x) { float y; asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x)); return y; }
// p sigma(p), and its derivative sigma (1 + p (1 - sigma)), sigma = 1 / (1 + exp(-p)).  Where sigma is below 2^-126 (p < -87.3)
// it is 0, and so are both, for any finite p: what is dropped is less than 2^-119.  1 - sigma = exp(-p) sigma, with exp(-p) kept
// finite so that it is 0 there, not infinity times 0.  (Both keep NaN, and give it for -infinity, where the formulas do.)
__device__ __forceinline__ float silu(float p) { return p * rcp(1.f + ex2(p * -1.4426950408889634f)); }
__device__ __forceinline__ float silu_slope(float p) {
    const float e = ex2(p * -1.4426950408889634f), s = rcp(1.f + e);
    return s * fmaf(p, fminf(e, 3.402823466e38f) * s, 1.f);
}

// A sequence: its number, and its first token and one past its last in the batch row.
struct Seq { int n, first, end; };
template <bool PACKED>
__device__ __forceinline__ Seq sequence_at(const ConvArgs& a, int b, int t) {
    if (!PACKED) return {b, 0, a.T};
    const mix::Span s = mix::span_of(a.cu, a.n_seqs, a.T, t);
    return {s.n, s.first, s.end};
}

template <typename T, int V>
__device__ __forceinline__ void load_row(float (&d)[V], const T* p, bool in) {
    Vec<T, V> r;
    if (in) r.load(p); else r.zero();
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] = r.get(v);
}
// the input at place `at` of sequence s (negative: out of its initial state)
template <typename T, int V>
__device__ __forceinline__ void load_input(float (&d)[V], const ConvArgs& a, const Seq& s, size_t row0, int at, int c) {
    if (at >= 0) load_row<T, V>(d, static_cast<const T*>(a.x) + (row0 + s.first + at) * a.ldx + c, true);
    else load_row<T, V>(d, static_cast<const T*>(a.h0) + ((size_t)s.n * (a.W - 1) + at + a.W - 1) * a.D + c, a.h0 != nullptr);
}

template <int W, int V>
struct Taps {
    float w[W][V], b[V];
    __device__ __forceinline__ void load(const ConvArgs& a, int c, bool live) {
        if (V == 4 && live && reinterpret_cast<uintptr_t>(a.w) % 16 == 0) {       // the channels' taps lie together
            float t[4 * W];
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float4 q = reinterpret_cast<const float4*>(a.w + (size_t)c * W)[i];
                t[4 * i] = q.x; t[4 * i + 1] = q.y; t[4 * i + 2] = q.z; t[4 * i + 3] = q.w;
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
#pragma unroll
                for (int j = 0; j < W; ++j) w[j][v] = t[(v * W + j) % (4 * W)];
                b[v] = a.b ? a.b[c + v] : 0.f;
            }
            return;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][v] = live ? a.w[(size_t)(c + v) * W + j] : 0.f;
            b[v] = live && a.b ? a.b[c + v] : 0.f;
        }
    }
};

// rows [N, W - 1] of the final states (forward) or of the initial states' gradients (backward), a warp each
template <typename T, int W, int V, bool BACKWARD>
__device__ __forceinline__ void state_row(const ConvArgs& a, int64_t r, int c) {
    const int n = (int)(r / (W - 1)), j = (int)(r % (W - 1));
    Seq s{n, 0, a.T};
    size_t row0 = (size_t)n * a.T;
    if (a.cu) {
        s.first = mix::clamp_off(a.cu[n], a.T);
        s.end = max(mix::clamp_off(a.cu[n + 1], a.T), s.first);
        row0 = 0;
    }
    const int len = s.end - s.first;
    Vec<T, V> o;
    if constexpr (!BACKWARD) {
        float d[V];
        load_input<T, V>(d, a, s, row0, len - (W - 1) + j, c);
#pragma unroll
        for (int v = 0; v < V; ++v) o.set(v, d[v]);
        o.store(static_cast<T*>(a.hT) + r * a.D + c);
    } else {
        // the input at place j - (W - 1) is tap j - t of token t
        Taps<W, V> k;
        k.load(a, c, true);
        float g[V] = {};
#pragma unroll
        for (int t = 0; t < W - 1; ++t) {
            if (t > j || t >= len) break;
            float p[V], dy[V];
#pragma unroll
            for (int v = 0; v < V; ++v) p[v] = k.b[v];
#pragma unroll
            for (int i = 0; i < W; ++i) {
                float x[V];
                load_input<T, V>(x, a, s, row0, t - (W - 1) + i, c);
#pragma unroll
                for (int v = 0; v < V; ++v) p[v] = fmaf(k.w[i][v], x[v], p[v]);
            }
            load_row<T, V>(dy, static_cast<const T*>(a.dy) + (row0 + s.first + t) * a.D + c, true);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float ds = a.silu ? dy[v] * silu_slope(p[v]) : dy[v];
                float w = 0.f;
#pragma unroll
                for (int i = 0; i < W; ++i) w = i == j - t ? k.w[i][v] : w;
                g[v] = fmaf(w, ds, g[v]);
            }
        }
        const int tail = j - len;                 // its place in the final state of a sequence shorter than that
        if (a.dhT && tail >= 0) {
            float d[V];
            load_row<T, V>(d, static_cast<const T*>(a.dhT) + ((size_t)n * (W - 1) + tail) * a.D + c, true);
#pragma unroll
            for (int v = 0; v < V; ++v) g[v] += d[v];
        }
#pragma unroll
        for (int v = 0; v < V; ++v) o.set(v, g[v]);
        o.store(static_cast<T*>(a.dh0) + r * a.D + c);
    }
}

// The grid: for every 32 V channels, the blocks of 8 runs (of whatever batch rows), then those of 8 state rows.
struct Grid { int cols, run, runs, run_blocks, state_blocks; };      // runs: of a batch row
// Tokens a run: as many as leave 32 warps of 128 channels for each of 152 SMs, since a run's neighbourhood is walked twice
// (65,536 packed tokens x 4096 channels: forward 185 us with 32 tokens and 172 with 64, backward 408 and 351; 128 gain
// nothing), and 16 where there are few.
int run_of(const ConvArgs& a) {
    for (int run = 64; run > 16; run /= 2)
        if ((int64_t)a.B * ((a.T + run - 1) / run) * ((a.D + 127) / 128) >= 152 * 32) return run;
    return 16;
}
Grid grid_of(const ConvArgs& a, int V, bool states) {
    const int run = run_of(a), runs = (a.T + run - 1) / run;
    const int64_t rows = (int64_t)a.N() * (a.W - 1);
    return {(a.D + 32 * V - 1) / (32 * V), run, runs, (int)(((int64_t)a.B * runs + kWarps - 1) / kWarps),
            states ? (int)((rows + kWarps - 1) / kWarps) : 0};
}

template <typename T, int W, int V, bool PACKED>
__global__ void __launch_bounds__(kThreads) conv_fwd_kernel(const ConvArgs a, const Grid g) {
    constexpr int kRing = kFwdRing;
    extern __shared__ __align__(16) unsigned char s_raw[];
    auto* ring = reinterpret_cast<Vec<T, V>*>(s_raw) + threadIdx.x;           // [kRing][256]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = ((int)(blockIdx.x % g.cols) * 32 + lane) * V;
    const int64_t block = blockIdx.x / g.cols;
    if (c >= a.D) return;
    if (block >= (int64_t)g.run_blocks) {
        const int64_t r = (block - (int64_t)g.run_blocks) * kWarps + warp;
        if (r < (int64_t)a.N() * (W - 1)) state_row<T, W, V, false>(a, r, c);
        return;
    }
    const int64_t r = block * kWarps + warp;
    if (r >= (int64_t)a.B * g.runs) return;
    const int b = (int)(r / g.runs), t0 = (int)(r % g.runs) * g.run;
    const int t1 = min(t0 + g.run, a.T);
    if (t0 >= t1) return;
    const size_t row0 = (size_t)b * a.T;
    const T* x = static_cast<const T*>(a.x) + (row0 + t0) * a.ldx + c;
    T* y = static_cast<T*>(a.y) + (row0 + t0) * a.D + c;
    Seq s = sequence_at<PACKED>(a, b, t0);
    float win[W - 1][V];                          // the last W - 1 inputs, oldest first
    Taps<W, V> k;
    // CLEAN: a whole run of one sequence, nothing to look out for
    const auto walk = [&](auto clean) {
        constexpr bool CLEAN = decltype(clean)::value;
        const auto fetch = [&](int t, int slot) {
            if (t < t1) {
#pragma unroll
                for (int i = 0; i < kChunk; ++i) {
                    const bool in = CLEAN || t + i < t1;
                    mix::copy_async(ring + (slot + i) * kThreads, in ? x : static_cast<const T*>(a.x), in);
                    x += a.ldx;
                }
            }
            mix::copies_close();
        };
#pragma unroll
        for (int m = 0; m < kRing; m += kChunk) fetch(t0 + m, m);
        k.load(a, c, true);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) load_input<T, V>(win[j], a, s, row0, t0 - s.first - (W - 1) + j, c);
        int slot = 0;
#pragma unroll 1
        for (int t = t0; t < t1; t += kChunk) {
            mix::copies_wait<kRing / kChunk - 1>();
#pragma unroll
            for (int i = 0; i < kChunk; ++i) {
                if (!CLEAN && t + i >= t1) break;
                if (!CLEAN && PACKED && t + i >= s.end) {
                    s = sequence_at<true>(a, b, t + i);
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) load_input<T, V>(win[j], a, s, row0, j - (W - 1), c);
                }
                const Vec<T, V> cur = ring[(slot + i) * kThreads];
                float xv[V], p[V];
#pragma unroll
                for (int v = 0; v < V; ++v) xv[v] = cur.get(v);
                mix::fma_row(p, k.w[W - 1], xv, k.b);
#pragma unroll
                for (int j = 0; j < W - 1; ++j) mix::fma_row(p, k.w[j], win[j], p);
                Vec<T, V> o;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    o.set(v, a.silu ? silu(p[v]) : p[v]);
#pragma unroll
                    for (int j = 0; j < W - 2; ++j) win[j][v] = win[j + 1][v];
                    win[W - 2][v] = xv[v];
                }
                o.store(y);
                y += a.D;
            }
            fetch(t + kRing, slot);
            slot = slot + kChunk == kRing ? 0 : slot + kChunk;
        }
    };
    if (t0 + g.run <= (PACKED ? min(s.end, a.T) : a.T)) walk(std::true_type{});
    else walk(std::false_type{});
}

template <typename T, int W, int V, bool PACKED>
__global__ void __launch_bounds__(kThreads, 2) conv_bwd_kernel(const ConvArgs a, const Grid g, float* part) {
    constexpr int kRing = kBwdRing;
    mix::let_next();
    extern __shared__ __align__(16) unsigned char s_raw[];
    auto* rx = reinterpret_cast<Vec<T, V>*>(s_raw) + threadIdx.x;             // [kRing][256] each
    auto* ry = rx + kRing * kThreads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = ((int)(blockIdx.x % g.cols) * 32 + lane) * V;
    const bool live = c < a.D;
    const int64_t block = blockIdx.x / g.cols;
    if (block >= (int64_t)g.run_blocks) {
        const int64_t r = (block - (int64_t)g.run_blocks) * kWarps + warp;
        if (live && r < (int64_t)a.N() * (W - 1)) state_row<T, W, V, true>(a, r, c);
        return;
    }
    const int64_t r = block * kWarps + warp;
    const bool run_there = r < (int64_t)a.B * g.runs;
    const int b = run_there ? (int)(r / g.runs) : 0, t0 = run_there ? (int)(r % g.runs) * g.run : a.T;
    const int t1 = live ? min(t0 + g.run, a.T) : t0;            // the run's tokens
    const int t2 = min(t1 + W - 1, a.T);                       // and those whose ds they need
    const size_t row0 = (size_t)b * a.T;
    float dw[W + 1][V];                                        // the taps', then the bias's
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) dw[j][v] = 0.f;
    if (t0 < t1) {
        const T* x = static_cast<const T*>(a.x) + (row0 + t0) * a.ldx + c;
        const T* dy = static_cast<const T*>(a.dy) + (row0 + t0) * a.D + c;
        T* dx = static_cast<T*>(a.dx) + (row0 + t0) * a.D + c;
        Taps<W, V> k;
        Seq s = sequence_at<PACKED>(a, b, t0);
        float win[W - 1][V], ds[W - 1][V];                     // the last W - 1 inputs and ds, oldest first
        int end[W - 1], own[W - 1];                            // the sequences of the last W - 1 tokens
        // CLEAN: a whole run of one sequence, and the tokens behind it that it needs too
        const auto walk = [&](auto clean) {
            constexpr bool CLEAN = decltype(clean)::value;
            const auto fetch = [&](int t, int slot) {
                if (t < t2) {
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) {
                        const bool in = t + i < t2;
                        mix::copy_async(rx + (slot + i) * kThreads, in ? x : static_cast<const T*>(a.x), in);
                        mix::copy_async(ry + (slot + i) * kThreads, in ? dy : static_cast<const T*>(a.dy), in);
                        x += a.ldx;
                        dy += a.D;
                    }
                }
                mix::copies_close();
            };
#pragma unroll
            for (int m = 0; m < kRing; m += kChunk) fetch(t0 + m, m);
            k.load(a, c, true);
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                load_input<T, V>(win[j], a, s, row0, t0 - s.first - (W - 1) + j, c);
                end[j] = s.end;
                own[j] = s.n;
#pragma unroll
                for (int v = 0; v < V; ++v) ds[j][v] = 0.f;
            }
            // Token `now` brings ds; dx of token now - (W - 1) is then complete.  INSIDE: the token is of the run (else
            // one behind it, whose ds the run's last tokens need; past the row's end ds is 0).
            const auto token = [&](int now, int at, auto inside) {
                constexpr bool INSIDE = decltype(inside)::value;
                const int out = now - (W - 1);
                if (!CLEAN && PACKED && now >= s.end && now < a.T) {
                    s = sequence_at<true>(a, b, now);
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) load_input<T, V>(win[j], a, s, row0, j - (W - 1), c);
                }
                float xv[V], p[V], d[V];
                const bool there = CLEAN || now < t2;          // (what is not was not copied)
                const Vec<T, V> cx = rx[at * kThreads], cy = ry[at * kThreads];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    xv[v] = there ? cx.get(v) : 0.f;
                    d[v] = there ? cy.get(v) : 0.f;
                }
                if (a.silu) {
                    mix::fma_row(p, k.w[W - 1], xv, k.b);
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) mix::fma_row(p, k.w[j], win[j], p);
#pragma unroll
                    for (int v = 0; v < V; ++v) p[v] = silu_slope(p[v]);
                    mix::mul_row(d, d, p);
                }
                if (!CLEAN && now >= a.T)
#pragma unroll
                    for (int v = 0; v < V; ++v) d[v] = 0.f;
                if (INSIDE) {
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) mix::fma_row(dw[j], d, win[j], dw[j]);
                    mix::fma_row(dw[W - 1], d, xv, dw[W - 1]);
#pragma unroll
                    for (int v = 0; v < V; ++v) dw[W][v] += d[v];
                }
                if (out >= t0) {
                    // ds at out .. out + reach - 1 belong to the token's sequence; that of out + m meets tap W - 1 - m
                    const int reach = CLEAN ? W : (PACKED ? end[0] : a.T) - out;
                    float gx[V];
                    mix::mul_row(gx, k.w[W - 1], ds[0]);
                    if (CLEAN || !PACKED || reach >= W) {
#pragma unroll
                        for (int m = 1; m < W - 1; ++m) mix::fma_row(gx, k.w[W - 1 - m], ds[m], gx);
                        mix::fma_row(gx, k.w[0], d, gx);
                    } else {
#pragma unroll
                        for (int m = 1; m < W - 1; ++m)
                            if (m < reach) mix::fma_row(gx, k.w[W - 1 - m], ds[m], gx);
                    }
                    const int tail = W - 1 - reach;            // its place in its sequence's final state
                    if (!CLEAN && a.dhT && tail >= 0) {
                        float e[V];
                        const int n = PACKED ? own[0] : b;
                        load_row<T, V>(e, static_cast<const T*>(a.dhT) + ((int64_t)n * (W - 1) + tail) * a.D + c, true);
#pragma unroll
                        for (int v = 0; v < V; ++v) gx[v] += e[v];
                    }
                    Vec<T, V> o;
#pragma unroll
                    for (int v = 0; v < V; ++v) o.set(v, gx[v]);
                    o.store(dx);
                    dx += a.D;
                }
#pragma unroll
                for (int j = 0; j < W - 2; ++j) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        win[j][v] = win[j + 1][v];
                        ds[j][v] = ds[j + 1][v];
                    }
                    end[j] = end[j + 1];
                    own[j] = own[j + 1];
                }
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    win[W - 2][v] = xv[v];
                    ds[W - 2][v] = d[v];
                }
                end[W - 2] = s.end;
                own[W - 2] = s.n;
            };
            int slot = 0, t = t0;
#pragma unroll 1
            for (; CLEAN ? t < t1 : t + kChunk <= t1; t += kChunk) {
                mix::copies_wait<kRing / kChunk - 1>();
#pragma unroll
                for (int i = 0; i < kChunk; ++i) token(t + i, slot + i, std::true_type{});
                fetch(t + kRing, slot);
                slot = slot + kChunk == kRing ? 0 : slot + kChunk;
            }
            mix::copies_wait<0>();
#pragma unroll 1
            for (; t < t1; ++t) {                              // (a row's end inside a group)
                token(t, slot, std::true_type{});
                slot = slot + 1 == kRing ? 0 : slot + 1;
            }
#pragma unroll 1
            for (; t < t1 + W - 1; ++t) {
                token(t, slot, std::false_type{});
                slot = slot + 1 == kRing ? 0 : slot + 1;
            }
        };
        if (t0 + g.run + W <= (PACKED ? min(s.end, a.T) : a.T)) walk(std::true_type{});
        else walk(std::false_type{});
    }
    mix::copies_wait<0>();
    __syncthreads();
    auto& sum = *reinterpret_cast<float(*)[kWarps][W + 1][32 * V]>(s_raw);     // (the rings are done with)
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) sum[warp][j][lane * V + v] = dw[j][v];
    __syncthreads();
    // part [W + 1][blocks][D]
    const int64_t rows = (int64_t)g.run_blocks;
    for (int i = threadIdx.x; i < (W + 1) * 32 * V; i += kWarps * 32) {
        const int j = i / (32 * V), lc = i % (32 * V), cc = (int)(blockIdx.x % g.cols) * 32 * V + lc;
        if (cc >= a.D) continue;
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) t += sum[w][j][lc];
        part[(j * rows + block) * a.D + cc] = t;
    }
}

// sums over the blocks: 32 channels a block, 8 row lanes, joined in order; blockIdx.y is the tap, or W for the bias
__global__ void __launch_bounds__(256) conv_param_kernel(const float* part, int64_t rows, int D, int W, float* dw, float* db) {
    __shared__ float s[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane, j = blockIdx.y;
    if (j == W && !db) return;
    mix::wait_behind();
    float acc = 0.f;
    if (c < D)
#pragma unroll 4
        for (int64_t r = w; r < rows; r += 8) acc += part[(j * rows + r) * D + c];
    s[w][lane] = acc;
    __syncthreads();
    if (w == 0 && c < D) {
        float t = 0.f;
        for (int i = 0; i < 8; ++i) t += s[i][lane];
        if (j < W) dw[(size_t)c * W + j] = t; else db[c] = t;
    }
}

// a thread takes V channels of up to `per` sequences, whose loads are under way together
constexpr int kStepSeqs = 4;
template <typename T, int W, int V>
__global__ void __launch_bounds__(128) conv_step_kernel(const ConvArgs a, const T* state, T* out, const int per) {
    const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int cols = a.D / V;
    const int64_t n0 = id / cols * per;
    const int c = (int)(id % cols) * V;
    if (n0 >= a.B) return;
    const int count = (int)min((int64_t)per, a.B - n0);
    Vec<T, V> win[kStepSeqs][W];
#pragma unroll
    for (int i = 0; i < kStepSeqs; ++i) {
        if (i >= count) break;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) win[i][j].load(state + ((n0 + i) * (W - 1) + j) * a.D + c);
        win[i][W - 1].load(static_cast<const T*>(a.x) + (n0 + i) * a.ldx + c);
    }
    Taps<W, V> k;
    k.load(a, c, true);
#pragma unroll
    for (int i = 0; i < kStepSeqs; ++i) {
        if (i >= count) break;
        Vec<T, V> y;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float p = k.b[v];
#pragma unroll
            for (int j = 0; j < W; ++j) p = fmaf(k.w[j][v], win[i][j].get(v), p);
            y.set(v, a.silu ? silu(p) : p);
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j) win[i][j + 1].store(out + ((n0 + i) * (W - 1) + j) * a.D + c);
        y.store(static_cast<T*>(a.y) + (n0 + i) * a.D + c);
    }
}

// Whether rows can be accessed V channels at a time (4 where they can, else 1: 16,384 tokens x 2048 channels 31 us and 50 us
// forward, 64 and 99 us backward).
bool vector_ok(const ConvArgs& a, int V, const void* state = nullptr, const void* state_out = nullptr) {
    const size_t bytes = V * (a.bf16 ? 2 : 4);
    const auto al = [&](const void* p) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; };
    return a.D % V == 0 && a.ldx % V == 0 && al(a.x) && al(a.h0) && al(a.hT) && al(a.y) && al(a.dy) && al(a.dhT) &&
           al(a.dx) && al(a.dh0) && al(state) && al(state_out);
}
cudaError_t allow_smem(const void* kernel, size_t bytes) {
    return bytes > 48 * 1024 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes)
                             : cudaSuccess;
}
template <typename F>
void by_width(int W, F f) {
    if (W == 2) f(std::integral_constant<int, 2>{});
    else if (W == 3) f(std::integral_constant<int, 3>{});
    else f(std::integral_constant<int, 4>{});
}
template <typename F>
void by_type(const ConvArgs& a, bool wide, F f) {
    const auto vec = [&](auto* t) {
        if (wide) f(t, std::integral_constant<int, 4>{});
        else f(t, std::integral_constant<int, 1>{});
    };
    if (a.bf16) vec((bf16*)nullptr);
    else vec((float*)nullptr);
}

}  // namespace

size_t conv_workspace_bytes(const ConvArgs& a) {
    return (size_t)grid_of(a, 1, false).run_blocks * (a.W + 1) * a.D * sizeof(float);
}

cudaError_t launch_conv_fwd(const ConvArgs& a, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    by_width(a.W, [&](auto w) {
        by_type(a, vector_ok(a, 4), [&](auto* t, auto v) {
            using T = std::remove_pointer_t<decltype(t)>;
            const Grid g = grid_of(a, v.value, a.hT != nullptr);
            const unsigned blocks = (unsigned)(g.cols * ((int64_t)g.run_blocks + g.state_blocks));
            if (blocks == 0) return;
            const size_t smem = (size_t)kFwdRing * kThreads * v.value * sizeof(T);
            const auto kernel = a.cu ? conv_fwd_kernel<T, w.value, v.value, true> : conv_fwd_kernel<T, w.value, v.value, false>;
            e = allow_smem(reinterpret_cast<const void*>(kernel), smem);
            if (e == cudaSuccess) kernel<<<blocks, kThreads, smem, s>>>(a, g);
        });
    });
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_conv_bwd(const ConvArgs& a, cudaStream_t s) {
    float* part = static_cast<float*>(a.ws);
    int64_t rows = 0;
    cudaError_t e = cudaSuccess;
    by_width(a.W, [&](auto w) {
        by_type(a, vector_ok(a, 4), [&](auto* t, auto v) {
            using T = std::remove_pointer_t<decltype(t)>;
            const Grid g = grid_of(a, v.value, a.dh0 != nullptr);
            rows = (int64_t)g.run_blocks;
            const unsigned blocks = (unsigned)(g.cols * (rows + g.state_blocks));
            if (blocks == 0) return;
            const size_t rings = 2 * (size_t)kBwdRing * kThreads * v.value * sizeof(T);
            const size_t sums = (size_t)kWarps * (w.value + 1) * 32 * v.value * sizeof(float);
            const size_t smem = rings > sums ? rings : sums;
            const auto kernel = a.cu ? conv_bwd_kernel<T, w.value, v.value, true> : conv_bwd_kernel<T, w.value, v.value, false>;
            e = allow_smem(reinterpret_cast<const void*>(kernel), smem);
            if (e == cudaSuccess) kernel<<<blocks, kThreads, smem, s>>>(a, g, part);
        });
    });
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return mix::launch_behind(conv_param_kernel, dim3((a.D + 31) / 32, a.W + 1), 256, 0, rows > 0, s, part, rows, a.D, a.W, a.dw,
                              a.db);
}

cudaError_t launch_conv_step(const ConvArgs& a, const void* state, void* state_out, cudaStream_t s) {
    by_width(a.W, [&](auto w) {
        by_type(a, vector_ok(a, 4, state, state_out), [&](auto* t, auto v) {
            using T = std::remove_pointer_t<decltype(t)>;
            // several sequences a thread once there are threads for every SM without (152 x 2048): 256 sequences x 6144 channels 10.9 us
            // so and 13.0 with one (both after an L2 flush)
            const int64_t cols = a.D / v.value;
            const int per = (int64_t)a.B * cols > 152 * 2048 ? kStepSeqs : 1;
            const int64_t threads = (a.B + per - 1) / per * cols;
            conv_step_kernel<T, w.value, v.value><<<(unsigned)((threads + 127) / 128), 128, 0, s>>>(
                a, static_cast<const T*>(state), static_cast<T*>(state_out), per);
        });
    });
    return cudaGetLastError();
}

}  // namespace gdn
