// Gated linear recurrence: scan forward, and the decode step.
//   h_t = a_t h_{t-1} + u_t,  o_t = h_t;  see glr_math.cuh for a and u, glr_scan.cuh for the tiling and the carry.
// x, g and in_gate are read once and o is written once (268 MB for B4 T4096 D2048 in bf16, 40 us at the copy rate).  Measured
// 82 us with both activations and the normalisation, 61 with the normalisation alone, 131 in fp32 (537 MB): at 60 instructions
// an element and about 2 instructions a cycle the kernel is bound by issue and by the latency of 12 warps an SM, not by HBM.  The shape of a block (16 lanes x 4 channels x 8 tokens, 32 elements a thread in
// registers) trades warps for instructions: runs of 4 tokens, 95 us.

#include <type_traits>

#include "glr_scan.cuh"
#include "internal.h"

namespace gdn {
namespace {

using namespace glr;
using mix::bf16;
using mix::Vec;

__device__ unsigned g_glr_status;   // bit 0: a block gave up a bounded wait

template <typename Tx, typename Tg, typename S, bool PACKED>
__global__ void __launch_bounds__(S::kBlock, 2)
glr_fwd_kernel(const GlrArgs a, const Exchange x, const int publish) {
    constexpr int LANES = S::LANES, V = S::V, W = S::W, R = S::R, L = S::L, kThreads = S::kThreads;
    static_assert(W <= kCarryThreads, "a carry thread for every channel");
    extern __shared__ __align__(16) unsigned char s_raw[];
    __shared__ float sA[2][R][W], sH[2][R][W];
    __shared__ int s_start[PACKED ? kPlaces : 1][kTile], s_end[PACKED ? kPlaces : 1][kTile];
    __shared__ bool s_marked[kPlaces][2];        // whether either half of a tile's tokens has a mark
    __shared__ __align__(16) Channel s_chan[kPlaces][W];
    __shared__ Tile s_tile[kPlaces];
    const int tid = threadIdx.x;
    mix::wait_behind();                          // for the clearing

    if (tid >= kThreads) {                       // the carry threads
        const int ch = tid - kThreads;
        const auto prepare = [&](int slot) {      // a place's channels and marks
            if (s_tile[slot].chain < 0) return;
            const int pc = tid - kThreads, c = s_tile[slot].c0 + pc;
            if (a.A_log && pc < W && c < a.D) s_chan[slot][pc] = channel(a.A_log, a.dt_bias, c);
            if (!PACKED) return;
            const bool any = sequence_marks(a, s_tile[slot].p, ch, s_start[slot], s_end[slot]);
            if (ch % 32 == 0) s_marked[slot][ch / 32] = any;
        };
        Tickets tickets(x);
        unsigned ticket = 0;
        first_tiles(x, a, W, false, tickets, s_tile, ch == 0, [] { __syncthreads(); });
        if (ch == 0) ticket = tickets.take();
        __syncwarp();
        S::sync(kMaps);                         // (places are read below by all carry threads: meet once)
        for (int i = 0; i < 3; ++i) prepare(i);
        __syncthreads();
        for (int i = 0; s_tile[i % kPlaces].chain >= 0; ++i) {
            const Tile t = s_tile[i % kPlaces];
            const int k = i & 1, ahead = (i + 3) % kPlaces;
            if (ch == 0) {
                s_tile[ahead] = tile_of(x, a, W, ticket, false);
                ticket = tickets.take();
            }
            float first = 0.f;
            if (!PACKED && ch < W && t.p < kSpan && a.h0 && t.c0 + ch < a.D) first = a.h0[(size_t)t.b * a.D + t.c0 + ch];
            S::sync(kMaps + k);
            if (ch < W) {
                // (a tile without marks forgets nothing inside)
                const bool marked = PACKED && (s_marked[i % kPlaces][0] || s_marked[i % kPlaces][1]);
                float A = 1.f, H = 0.f;
                if (marked) {
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        H = apply<true>(sA[k][r][ch], sH[k][r][ch], H);
                        A = both<true>(A, sA[k][r][ch]);
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        H = fmaf(sA[k][r][ch], H, sH[k][r][ch]);
                        A *= sA[k][r][ch];
                    }
                }
                float h = carry_in<PACKED>(x, W, t.p, t.chain, ch, A, H, first, publish || t.p > 0, &g_glr_status);
                if (a.ckpt && t.c0 + ch < a.D && t.p * kTile < a.T)
                    a.ckpt[((size_t)t.b * x.tiles + t.p) * a.D + t.c0 + ch] = h;
                if (marked) {
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float rH = sH[k][r][ch];
                        sH[k][r][ch] = h;
                        h = apply<true>(sA[k][r][ch], rH, h);
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float rH = sH[k][r][ch];
                        sH[k][r][ch] = h;
                        h = fmaf(sA[k][r][ch], h, rH);
                    }
                }
            }
            S::arrive(kCarry + k);
            prepare(ahead);
        }
        return;
    }

    // the compute threads
    const int run = tid / LANES, lane = tid % LANES, arrays = a.gi ? 3 : 2;
    const int bytes = L * kThreads * (int)(sizeof(Vec<Tg, V>) + (arrays - 1) * sizeof(Vec<Tx, V>));
    const auto buf_g = [&](int k) { return reinterpret_cast<Vec<Tg, V>*>(s_raw + k * bytes) + tid; };   // [L][kThreads] each
    const auto buf_x = [&](int k) {
        return reinterpret_cast<Vec<Tx, V>*>(s_raw + k * bytes + L * kThreads * sizeof(Vec<Tg, V>)) + tid;
    };
    const auto fetch = [&](int i) {
        const Tile t = s_tile[i % kPlaces];
        const int c = t.c0 + lane * V, t0 = t.p * kTile + run * L;
        const int n = t.chain >= 0 && c < a.D ? min(a.T - t0, L) : 0;
        const size_t row = (size_t)t.b * a.T + t0;
        const Tg* g = static_cast<const Tg*>(a.g) + row * a.ldg + c;
        const Tx* xp = static_cast<const Tx*>(a.x) + row * a.ldx + c;
        const Tx* ip = static_cast<const Tx*>(a.gi) + row * a.ldi + c;
        Vec<Tg, V>* bg = buf_g(i & 1);
        Vec<Tx, V>* bx = buf_x(i & 1);
        if (n == L) {
#pragma unroll
            for (int j = 0; j < L; ++j) {
                mix::copy_async(bg + j * kThreads, g, true);
                mix::copy_async(bx + j * kThreads, xp, true);
                if (a.gi) mix::copy_async(bx + (L + j) * kThreads, ip, true);
                g += a.ldg;
                xp += a.ldx;
                ip += a.ldi;
            }
            mix::copies_close();
            return;
        }
#pragma unroll 1
        for (int j = 0; j < L; ++j) {            // the row's end, or no channels
            mix::copy_async(bg + j * kThreads, j < n ? g : static_cast<const Tg*>(a.g), j < n);
            mix::copy_async(bx + j * kThreads, j < n ? xp : static_cast<const Tx*>(a.x), j < n);
            if (a.gi) mix::copy_async(bx + (L + j) * kThreads, j < n ? ip : static_cast<const Tx*>(a.gi), j < n);
            g += a.ldg;
            xp += a.ldx;
            ip += a.ldi;
        }
        mix::copies_close();
    };
    const auto run_starts = [&](int i) {         // which tokens of the run start a sequence
        unsigned m = 0;
#pragma unroll
        for (int j = 0; j < L; ++j) m |= (s_start[i % kPlaces][run * L + j] >= 0 ? 1u : 0u) << j;
        return m;
    };

    // stage one: decays and inputs of the run, and its map
    const auto maps = [&](int i, float (&al)[L][V], float (&u)[L][V]) {
        const Tile t = s_tile[i % kPlaces];
        const int c = t.c0 + lane * V, count = a.T - (t.p * kTile + run * L);
        const bool live = c < a.D;
        const Vec<Tg, V>* bg = buf_g(i & 1);
        const Vec<Tx, V>* bx = buf_x(i & 1);
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const Vec<Tg, V> g = bg[j * kThreads];
            const Vec<Tx, V> xv = bx[j * kThreads];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                al[j][v] = g.get(v);
                u[j][v] = xv.get(v);
            }
        }
        if (a.gi) {
#pragma unroll
            for (int j = 0; j < L; ++j) {
                const Vec<Tx, V> gi = bx[(L + j) * kThreads];
#pragma unroll
                for (int v = 0; v < V; ++v) u[j][v] *= sigmoid(gi.get(v));
            }
        }
        log_decays<L, V>(a, s_chan[i % kPlaces] + lane * V, al);
        decays<L, V>(al, [&](int j, int v, const auto&... d) {
            if (a.normalize) {
                float power[sizeof...(d)];
                input_powers(power, d...);
                times_factors<sizeof...(d)>(&u[j][v], power);
            }
            ((al[j][v++] = d.a), ...);
        });
        if (count < L) {                         // past the row's end the state stays
#pragma unroll
            for (int j = 0; j < L; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) al[j][v] = j < count ? al[j][v] : 1.f;
        }
        float A[V], H[V];
        const unsigned starts = PACKED && (s_marked[i % kPlaces][0] || s_marked[i % kPlaces][1]) ? run_starts(i) : 0;
        if (PACKED && starts) {
#pragma unroll
            for (int j = 0; j < L; ++j) {
                const bool here = (starts >> j) & 1;
                if (here && a.h0 && live) {
                    const float* h0 = a.h0 + (size_t)s_start[i % kPlaces][run * L + j] * a.D + c;
#pragma unroll
                    for (int v = 0; v < V; ++v) u[j][v] = fmaf(al[j][v], h0[v], u[j][v]);
                }
#pragma unroll
                for (int v = 0; v < V; ++v) H[v] = here || j == 0 ? u[j][v] : fmaf(al[j][v], H[v], u[j][v]);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) A[v] = -1.f;
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                H[v] = u[0][v];
                A[v] = al[0][v];
            }
#pragma unroll
            for (int j = 1; j < L; ++j) {
                mix::fma_row(H, al[j], H, u[j]);
                mix::mul_row(A, A, al[j]);
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            sA[i & 1][run][lane * V + v] = A[v];
            sH[i & 1][run][lane * V + v] = H[v];
        }
        S::arrive(kMaps + (i & 1));
    };

    // stage two: the states
    const auto states = [&](int i, const float (&al)[L][V], const float (&u)[L][V]) {
        const Tile t = s_tile[i % kPlaces];
        const int c = t.c0 + lane * V, t0 = t.p * kTile + run * L;
        const bool live = c < a.D;
        float h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = sH[i & 1][run][lane * V + v];
        Tx* op = static_cast<Tx*>(a.o) + ((size_t)t.b * a.T + t0) * a.D + c;
        const int n = live && a.o ? a.T - t0 : 0;
        if (PACKED && (s_marked[i % kPlaces][0] || s_marked[i % kPlaces][1])) {
            const unsigned starts = run_starts(i);
#pragma unroll
            for (int j = 0; j < L; ++j) {
                Vec<Tx, V> o;
                const bool here = (starts >> j) & 1;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    h[v] = here ? u[j][v] : fmaf(al[j][v], h[v], u[j][v]);
                    o.set(v, h[v]);
                }
                if (j < n) o.store(op);
                op += a.D;
                const int m = s_end[i % kPlaces][run * L + j];
                if (a.hT && live && m >= 0)
#pragma unroll
                    for (int v = 0; v < V; ++v) a.hT[(size_t)m * a.D + c + v] = h[v];
            }
        } else {
#pragma unroll
            for (int j = 0; j < L; ++j) {
                Vec<Tx, V> o;
                mix::fma_row(h, al[j], h, u[j]);
#pragma unroll
                for (int v = 0; v < V; ++v) o.set(v, h[v]);
                if (j < n) o.store(op);
                op += a.D;
            }
        }
        if (!PACKED && a.hT && live && t.p == x.tiles - 1 && run == R - 1)
#pragma unroll
            for (int v = 0; v < V; ++v) a.hT[(size_t)t.b * a.D + c + v] = h[v];
        if (PACKED && a.hT && live) {
            // empty sequences end as they began; the row's tiles share them
            for (int m = t.p * R + run; m < a.n_seqs; m += x.tiles * R) {
                if (mix::clamp_off(a.cu[m + 1], a.T) > mix::clamp_off(a.cu[m], a.T)) continue;
#pragma unroll
                for (int v = 0; v < V; ++v) a.hT[(size_t)m * a.D + c + v] = a.h0 ? a.h0[(size_t)m * a.D + c + v] : 0.f;
            }
        }
    };

    __syncthreads();
    fetch(0);
    S::arrive(kMaps);
    __syncthreads();
    if (s_tile[0].chain < 0) return;
    fetch(1);
    float al[L][V], u[L][V], al_p[L][V], u_p[L][V];           // the current tile's, and the one's before it
    for (int i = 0;; ++i) {
        const bool more = s_tile[i % kPlaces].chain >= 0;
        if (more) {
            mix::copies_wait<1>();
            maps(i, al, u);
        }
        if (i > 0) S::sync(kCarry + ((i - 1) & 1));
        if (more) fetch(i + 2);
        if (i > 0) states(i - 1, al_p, u_p);
        if (!more) break;
#pragma unroll
        for (int j = 0; j < L; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                al_p[j][v] = al[j][v];
                u_p[j][v] = u[j][v];
            }
    }
}

__global__ void __launch_bounds__(256) glr_clear_kernel(uint4* p, size_t n) {
    mix::let_next();
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256)
        p[i] = make_uint4(kEmpty, kEmpty, kEmpty, kEmpty);
}

template <typename Tx, typename Tg>
__global__ void glr_step_kernel(const GlrStepArgs a) {
    const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t n = id / a.D;
    const int c = (int)(id % a.D);
    if (n >= a.N) return;
    const float g = mix::ld(static_cast<const Tg*>(a.g) + n * a.ldg + c);
    const Channel ch = channel(a.A_log, a.dt_bias, c);
    float la = a.A_log ? ch.neg_eA * softplus(g + ch.dt, tail(g + ch.dt)) : min_nan(g, 88.f);
    const Decay d = decay(la);
    float u = mix::ld(static_cast<const Tx*>(a.x) + n * a.ldx + c);
    if (a.normalize) {
        float power;
        input_powers(&power, d);
        times_factors<1>(&u, &power);
    }
    if (a.gi) u *= sigmoid(mix::ld(static_cast<const Tx*>(a.gi) + n * a.ldi + c));
    const float h = fmaf(d.a, a.h[n * a.D + c], u);
    a.h_out[n * a.D + c] = h;
    mix::st(static_cast<Tx*>(a.o) + n * a.D + c, h);
}

template <typename Tx, typename Tg, typename S, bool PACKED>
cudaError_t fwd(const GlrArgs& a, cudaStream_t s) {
    const Layout l = layout(a.B, a.T, a.D, S::W);
    const Exchange x = exchange(l, a.ws);
    if (l.bytes) {
        const cudaError_t e = clear(a.ws, l.bytes, s);
        if (e != cudaSuccess) return e;
    }
    const auto kernel = glr_fwd_kernel<Tx, Tg, S, PACKED>;
    const int smem = 2 * S::L * S::kThreads * S::V * (int)(sizeof(Tg) + (a.gi ? 2 : 1) * sizeof(Tx));
    static Residency res[2];                     // without and with the input gate
    int blocks = 0;
    const cudaError_t e = res[a.gi != nullptr].get(reinterpret_cast<const void*>(kernel), S::kBlock, smem, &blocks);
    if (e != cudaSuccess) return e;
    return mix::launch_behind(kernel, x.total < blocks ? x.total : blocks, S::kBlock, smem, l.bytes > 0, s, a, x,
                              a.test_stall ? 0 : 1);
}

template <typename Tx, typename Tg, typename S>
cudaError_t fwd_packed(const GlrArgs& a, cudaStream_t s) {
    return a.cu ? fwd<Tx, Tg, S, true>(a, s) : fwd<Tx, Tg, S, false>(a, s);
}

template <typename Tx, typename Tg>
cudaError_t fwd_wide(const GlrArgs& a, cudaStream_t s) {
    if (glr_vector(a, 4)) return fwd_packed<Tx, Tg, Shape<16, 4, 8>>(a, s);
    if (glr_vector(a, 2)) return fwd_packed<Tx, Tg, Shape<32, 2, 8>>(a, s);
    return fwd_packed<Tx, Tg, Shape<32, 1, 8>>(a, s);
}

}  // namespace

namespace glr {
cudaError_t clear(void* ws, size_t bytes, cudaStream_t s) {
    const size_t n = bytes / sizeof(uint4), blocks = (n + 1023) / 1024, most = 152 * 8;
    glr_clear_kernel<<<(unsigned)(blocks < most ? blocks : most), 256, 0, s>>>(static_cast<uint4*>(ws), n);
    return cudaGetLastError();
}
}  // namespace glr

// Whether rows can be read and written V channels at a time.  The widest access that everything is aligned to is taken
// (B4 T4096 D2048 in bf16: after a flush of L2: forward 87, 102 and 142 us with 4, 2 and 1; backward 199 us with 2, 258 with 1).
bool glr_vector(const GlrArgs& a, int V) {
    const size_t es = a.bf16 ? 2 : 4, gs = a.g_bf16 ? 2 : 4;
    const auto ok = [V](const void* p, size_t size) { return reinterpret_cast<uintptr_t>(p) % (V * size) == 0; };
    return a.D % V == 0 && a.ldx % V == 0 && a.ldg % V == 0 && (!a.gi || a.ldi % V == 0) && ok(a.x, es) && ok(a.g, gs) &&
           ok(a.gi, es) && ok(a.o, es) && ok(a.dO, es) && ok(a.dx, es) && ok(a.dg, gs) && ok(a.di, es);
}

cudaError_t launch_glr_fwd(const GlrArgs& a, cudaStream_t s) {
    if (!a.bf16) return fwd_wide<float, float>(a, s);
    return a.g_bf16 ? fwd_wide<bf16, bf16>(a, s) : fwd_wide<bf16, float>(a, s);
}

cudaError_t launch_glr_step(const GlrStepArgs& a, cudaStream_t s) {
    const unsigned blocks = (unsigned)(((int64_t)a.N * a.D + 127) / 128);
    if (!a.bf16) glr_step_kernel<float, float><<<blocks, 128, 0, s>>>(a);
    else if (a.g_bf16) glr_step_kernel<bf16, bf16><<<blocks, 128, 0, s>>>(a);
    else glr_step_kernel<bf16, float><<<blocks, 128, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t glr_read_and_clear_status(unsigned* value, bool clear) {
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return e;
    e = cudaMemcpyFromSymbol(value, g_glr_status, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_glr_status, &zero, sizeof(unsigned));
}

}  // namespace gdn
