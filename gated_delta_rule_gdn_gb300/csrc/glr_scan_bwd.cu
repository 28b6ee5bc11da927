// Backward of the gated linear recurrence, one pass over the tokens from the last to the first.
//   D_t = dO_t + G_{t+1},  G_t = a_t D_t  (G flows into h_{t-1}; after a sequence's last token it is dhT), and the chain of
//   each token's log a, s and sigma(i) with h_{t-1}.
// A block takes a tile as the forward does.  The states inside it come from the forward's checkpoint at its entry, by
// the same recurrence; G is carried between tiles in reverse (glr_scan.cuh).  So x, g, in_gate and dO are read once and
// the three gradients written once.  The per-channel sums of A_log and dt_bias leave the block as a row of partial sums
// that a second kernel adds in order.

#include "glr_scan.cuh"

namespace gdn {
namespace {

using namespace glr;
using mix::bf16;
using mix::Vec;

__device__ unsigned g_glr_bwd_status;   // bit 0: a block gave up a bounded wait

struct BwdSpace { void* scan; float* part; };

template <typename Tx, typename Tg, int LANES, int V, bool PACKED>
__global__ void __launch_bounds__(kThreads, 2)
glr_bwd_kernel(const GlrArgs a, const Exchange x, float* part) {
    using At = Place<LANES, V>;
    constexpr int W = At::W, R = At::kRuns, L = At::L;
    static_assert(2 * W <= kThreads, "one thread a channel for each direction");
    extern __shared__ __align__(16) unsigned char s_raw[];
    __shared__ float sA[R][W], sH[R][W], sG[R][W];
    __shared__ unsigned char s_any[R];           // bit 0: a sequence starts in the run; bit 1: one ends
    __shared__ int s_start[2][kTile], s_end[2][kTile];
    __shared__ unsigned s_next;
    const int tid = threadIdx.x, run = tid / LANES, lane = tid % LANES;
    auto* bg = reinterpret_cast<Vec<Tg, V>*>(s_raw) + tid;                    // [L][256] each
    auto* bx = reinterpret_cast<Vec<Tx, V>*>(s_raw + L * kThreads * sizeof(Vec<Tg, V>)) + tid;
    auto* bi = bx + L * kThreads;
    auto* bo = bi + L * kThreads;

    At at;
    const auto fetch = [&](int id) {
        at.set(x, a, id, true);
        const Tg* g = static_cast<const Tg*>(a.g) + at.row * a.ldg + at.c;
        const Tx* xp = static_cast<const Tx*>(a.x) + at.row * a.ldx + at.c;
        const Tx* ip = static_cast<const Tx*>(a.gi) + at.row * a.ldi + at.c;
        const Tx* op = static_cast<const Tx*>(a.dO) + at.row * a.D + at.c;
        const int n = at.live ? at.count : 0;
#pragma unroll
        for (int j = 0; j < L; ++j) {
            mix::copy_async(bg + j * kThreads, j < n ? g : static_cast<const Tg*>(a.g), j < n);
            mix::copy_async(bx + j * kThreads, j < n ? xp : static_cast<const Tx*>(a.x), j < n);
            if (a.gi) mix::copy_async(bi + j * kThreads, j < n ? ip : static_cast<const Tx*>(a.gi), j < n);
            mix::copy_async(bo + j * kThreads, j < n ? op : static_cast<const Tx*>(a.dO), j < n);
            g += a.ldg;
            xp += a.ldx;
            ip += a.ldi;
            op += a.D;
        }
        mix::copies_close();
    };
    // the state that enters the tile, for the threads that run the states through it (tid - W is their channel)
    const auto entry_state = [&]() {
        const int c = at.c0 + tid - W;
        if (tid < W || tid >= 2 * W || c >= a.D || at.p * kTile >= a.T) return 0.f;
        if (at.p > 0 || PACKED) return a.ckpt[((size_t)at.b * x.tiles + at.p) * a.D + c];
        return a.h0 ? a.h0[(size_t)at.b * a.D + c] : 0.f;
    };
    unsigned ticket = 0;
    int id = blockIdx.x;
    if (x.tiles > 1) {
        if (tid == 0) s_next = atomicAdd(x.ticket, 1u) + 1u;
        __syncthreads();
        id = (int)s_next;
        if (tid == 0) ticket = atomicAdd(x.ticket, 1u) + 1u;
        __syncthreads();
    }
    float entry = 0.f;
    if (id < x.total) {
        fetch(id);
        entry = entry_state();
        if (PACKED && tid < kTile) sequence_marks(a, at.p, s_start[0], s_end[0]);
    }
    if (PACKED) __syncthreads();

    for (int k = 0; id < x.total; k ^= 1) {
        const At now = at;
        unsigned starts = 0, ends = 0;
        if (PACKED) {
#pragma unroll
            for (int j = 0; j < L; ++j) {
                starts |= (s_start[k][run * L + j] >= 0 ? 1u : 0u) << j;
                ends |= (s_end[k][run * L + j] >= 0 ? 1u : 0u) << j;
            }
        }
        // the decay, the input u, and the factors of the gradients:
        //   dx = D w, di = dx y, dla = D (a h_{t-1} - m), dg = dla w3, dA_log = sum dla la
        //   w = s sigma(i), y = x (1 - sigma(i)), m = sigma(i) x a^2 / s, w3 = dla/dg
        float al[L][V], u[L][V], w[L][V], y[L][V], m[L][V], w3[L][V], la[L][V], dO[L][V];
        mix::copies_wait<0>();
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const Vec<Tg, V> g = bg[j * kThreads];
            const Vec<Tx, V> xv = bx[j * kThreads], ov = bo[j * kThreads];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                la[j][v] = g.get(v);
                u[j][v] = xv.get(v);
                dO[j][v] = ov.get(v);
                w[j][v] = w3[j][v] = 1.f;
                y[j][v] = m[j][v] = 0.f;
            }
        }
        if (a.gi) {
#pragma unroll
            for (int j = 0; j < L; ++j) {
                const Vec<Tx, V> gi = bi[j * kThreads];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    // 1 - sigma(i) = e sigma(i) with e = exp(-i), kept finite
                    const float e = ex2(max_nan(gi.get(v), -80.f) * -kLog2e), si = rcp(1.f + e);
                    w[j][v] = si;
                    u[j][v] *= si;
                    y[j][v] = u[j][v] * e;
                }
            }
        }
        if (a.A_log) {
            Channel ch[V];
#pragma unroll
            for (int v = 0; v < V; ++v) ch[v] = now.live ? channel(a.A_log, a.dt_bias, now.c + v) : Channel{0.f, 0.f};
#pragma unroll
            for (int j = 0; j < L; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float z = la[j][v] + ch[v].dt, e = tail(z);
                    la[j][v] = ch[v].neg_eA * softplus(z, e);
                    w3[j][v] = ch[v].neg_eA * sigmoid(z, e);
                }
        } else {
#pragma unroll
            for (int j = 0; j < L; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) la[j][v] = min_nan(la[j][v], 88.f);
        }
#pragma unroll
        for (int j = 0; j < L; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Decay d = decay(la[j][v]);
                if (a.normalize) {
                    // ds/dlog a = -a^2 / s, taken as 0 where s = 0 (log a = 0: the derivative does not exist there)
                    const float s2 = input_power(d), rs = s2 > 0.f ? rsq(s2) : 0.f, s = s2 * rs;
                    m[j][v] = u[j][v] * (d.a * d.a) * rs;
                    u[j][v] *= s;
                    w[j][v] *= s;
                }
                al[j][v] = d.a;
            }
        if (now.count < L) {                     // past the row's end state and gradient stay
#pragma unroll
            for (int j = 0; j < L; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) al[j][v] = j < now.count ? al[j][v] : 1.f;
        }
        if (PACKED && (starts | ends) && now.live) {
            // what enters at a sequence's first token, and at its last
#pragma unroll
            for (int j = 0; j < L; ++j) {
                if (((starts >> j) & 1) && a.h0)
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        u[j][v] = fmaf(al[j][v], a.h0[(size_t)s_start[k][run * L + j] * a.D + now.c + v], u[j][v]);
                if (((ends >> j) & 1) && a.dhT)
#pragma unroll
                    for (int v = 0; v < V; ++v) dO[j][v] += a.dhT[(size_t)s_end[k][run * L + j] * a.D + now.c + v];
            }
        }

        // the run's maps: (A, H) of the state, (A, G) of the gradient; one A serves both
        float A[V], H[V], G[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            A[v] = 1.f;
            H[v] = G[v] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const int r = L - 1 - j;
            const bool start = PACKED && ((starts >> j) & 1), end = PACKED && ((ends >> r) & 1);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                H[v] = start ? u[j][v] : fmaf(al[j][v], H[v], u[j][v]);
                G[v] = al[r][v] * (end ? dO[r][v] : dO[r][v] + G[v]);
                A[v] *= al[j][v];
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            sA[run][lane * V + v] = A[v];
            sH[run][lane * V + v] = H[v];
            sG[run][lane * V + v] = G[v];
        }
        if (PACKED && lane == 0) s_any[run] = (starts ? 1 : 0) | (ends ? 2 : 0);
        const float enter = entry;
        if (x.tiles > 1 && tid == 0) s_next = ticket;
        __syncthreads();
        const int next = x.tiles > 1 ? (int)s_next : id + (int)gridDim.x;
        if (next < x.total) {                    // the buffer is free: the next tile's inputs on the way
            fetch(next);
            entry = entry_state();
            if (PACKED && tid < kTile) sequence_marks(a, at.p, s_start[k ^ 1], s_end[k ^ 1]);
            if (x.tiles > 1 && tid == 0) ticket = atomicAdd(x.ticket, 1u) + 1u;
        }
        if (tid < W) {                           // the gradient that enters the tile from behind, and each of its runs
            const int c = now.c0 + tid;
            const auto run_A = [&](int r) { return PACKED && (s_any[r] & 2) ? -1.f : sA[r][tid]; };
            float tA = 1.f, tG = 0.f, G = 0.f;
#pragma unroll
            for (int r = R - 1; r >= 0; --r) {
                tG = apply(run_A(r), sG[r][tid], tG);
                tA = both(tA, run_A(r));
            }
            const int q = x.tiles - 1 - now.p;
            if (!PACKED && q < kGroup && a.dhT && c < a.D) G = a.dhT[(size_t)now.b * a.D + c];
            G = carry_in(x, W, q, now.chain, tid, tA, tG, G, true, &g_glr_bwd_status);
#pragma unroll
            for (int r = R - 1; r >= 0; --r) {
                const float rG = sG[r][tid];
                sG[r][tid] = G;
                G = apply(run_A(r), rG, G);
            }
        } else if (tid < 2 * W) {                // the states that enter the runs
            const int c = tid - W;
            float h = enter;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float rA = PACKED && (s_any[r] & 1) ? -1.f : sA[r][c], rH = sH[r][c];
                sH[r][c] = h;
                h = apply(rA, rH, h);
            }
        }
        __syncthreads();

        // h_{t-1} of every token in place of u, then the gradients from the last token to the first
        float h[V], pA[V], pdt[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            h[v] = sH[run][lane * V + v];
            G[v] = sG[run][lane * V + v];
            pA[v] = pdt[v] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const bool start = PACKED && ((starts >> j) & 1);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float uj = u[j][v];
                u[j][v] = h[v];
                if (start) {
                    u[j][v] = a.h0 && now.live ? a.h0[(size_t)s_start[k][run * L + j] * a.D + now.c + v] : 0.f;
                    h[v] = uj;
                } else {
                    h[v] = fmaf(al[j][v], h[v], uj);
                }
            }
        }
        Tx* dx_p = static_cast<Tx*>(a.dx) + (now.row + L) * a.D + now.c;
        Tx* di_p = static_cast<Tx*>(a.di) + (now.row + L) * a.D + now.c;
        Tg* dg_p = static_cast<Tg*>(a.dg) + (now.row + L) * a.D + now.c;
        const int n = now.live ? now.count : 0;
#pragma unroll
        for (int j = L - 1; j >= 0; --j) {
            const bool end = PACKED && ((ends >> j) & 1);
            Vec<Tx, V> dx, di;
            Vec<Tg, V> dg;
            dx_p -= a.D;
            di_p -= a.D;
            dg_p -= a.D;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float D = end ? dO[j][v] : dO[j][v] + G[v];
                G[v] = al[j][v] * D;
                const float dla = D * fmaf(al[j][v], u[j][v], -m[j][v]), dw = D * w[j][v], dz = dla * w3[j][v];
                dx.set(v, dw);
                di.set(v, dw * y[j][v]);
                dg.set(v, dz);
                if (j < n) {
                    pA[v] = fmaf(dla, la[j][v], pA[v]);
                    pdt[v] += dz;
                }
            }
            if (j < n) {
                dx.store(dx_p);
                dg.store(dg_p);
                if (a.gi) di.store(di_p);
            }
            if (PACKED && a.dh0 && now.live) {
                const int s = s_start[k][run * L + j];
                if (s >= 0)
#pragma unroll
                    for (int v = 0; v < V; ++v) a.dh0[(size_t)s * a.D + now.c + v] = G[v];
            }
        }
        if (!PACKED && a.dh0 && now.live && now.p == 0 && run == 0)
#pragma unroll
            for (int v = 0; v < V; ++v) a.dh0[(size_t)now.b * a.D + now.c + v] = G[v];
        if (PACKED && a.dh0 && now.live) {
            for (int s = now.p * R + run; s < a.n_seqs; s += x.tiles * R) {
                if (mix::clamp_off(a.cu[s + 1], a.T) > mix::clamp_off(a.cu[s], a.T)) continue;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    a.dh0[(size_t)s * a.D + now.c + v] = a.dhT ? a.dhT[(size_t)s * a.D + now.c + v] : 0.f;
            }
        }
        if (a.dA) {                              // the tile's sums, runs in order
#pragma unroll
            for (int v = 0; v < V; ++v) {
                sA[run][lane * V + v] = pA[v];
                sG[run][lane * V + v] = pdt[v];  // (each thread overwrites what it alone has read)
            }
            __syncthreads();
            if (tid < 2 * W && now.c0 + tid % W < a.D) {
                const float(*src)[W] = tid < W ? sA : sG;
                float s = 0.f;
#pragma unroll
                for (int r = 0; r < R; ++r) s += src[r][tid % W];
                const size_t rows = (size_t)a.B * x.tiles, r = (size_t)now.b * x.tiles + now.p;
                part[((tid < W ? 0 : rows) + r) * a.D + now.c0 + tid % W] = s;
            }
            __syncthreads();
        }
        id = next;
    }
}

// column sums of part [2][rows][D]: 32 channels a block, 8 row lanes, joined in order
__global__ void __launch_bounds__(256) glr_param_kernel(const float* part, int rows, int D, float* dA, float* ddt) {
    __shared__ float s[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    const float* src = part + (size_t)blockIdx.y * rows * D;
    float* out = blockIdx.y ? ddt : dA;
    if (!out) return;
    float acc[4] = {};
    if (c < D) {
        int r = w;
        for (; r + 24 < rows; r += 32)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] += src[(size_t)(r + 8 * i) * D + c];
        for (; r < rows; r += 8) acc[0] += src[(size_t)r * D + c];
    }
    s[w][lane] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
    __syncthreads();
    if (w == 0 && c < D) {
        float t = 0.f;
        for (int i = 0; i < 8; ++i) t += s[i][lane];
        out[c] = t;
    }
}

template <typename Tx, typename Tg, int LANES, int V, bool PACKED>
cudaError_t bwd(const GlrArgs& a, const BwdSpace& sp, cudaStream_t s) {
    using At = Place<LANES, V>;
    const Layout l = layout(a.B, a.T, a.D, At::W);
    const Exchange x = exchange(l, sp.scan);
    if (l.bytes) {
        const cudaError_t e = cudaMemsetAsync(sp.scan, 0xff, l.bytes, s);
        if (e != cudaSuccess) return e;
    }
    const auto kernel = glr_bwd_kernel<Tx, Tg, LANES, V, PACKED>;
    const size_t smem = (size_t)At::L * kThreads * V * (sizeof(Tg) + 3 * sizeof(Tx));
    static const Residency res = residency(reinterpret_cast<const void*>(kernel), smem);
    if (res.error != cudaSuccess) return res.error;
    kernel<<<x.total < res.blocks ? x.total : res.blocks, kThreads, smem, s>>>(a, x, sp.part);
    if (a.dA)
        glr_param_kernel<<<dim3((a.D + 31) / 32, 2), 256, 0, s>>>(sp.part, a.B * l.tiles, a.D, a.dA, a.ddt);
    return cudaGetLastError();
}

template <typename Tx, typename Tg, int LANES, int V>
cudaError_t bwd_packed(const GlrArgs& a, const BwdSpace& sp, cudaStream_t s) {
    return a.cu ? bwd<Tx, Tg, LANES, V, true>(a, sp, s) : bwd<Tx, Tg, LANES, V, false>(a, sp, s);
}

template <typename Tx, typename Tg>
cudaError_t bwd_wide(const GlrArgs& a, const BwdSpace& sp, cudaStream_t s) {
    if (glr_vector(a, 2)) return bwd_packed<Tx, Tg, 16, 2>(a, sp, s);
    return bwd_packed<Tx, Tg, 32, 1>(a, sp, s);
}

// The backward's workspace: the scan's exchange, the partial sums of the parameters, and the checkpoints that the
// caller did not keep (with the forward's exchange for computing them in the scan's place).
size_t up(size_t v) { return (v + 255) / 256 * 256; }
int tiles_of(const GlrArgs& a) { return layout(a.B, a.T, a.D, 32).tiles; }
size_t part_bytes(const GlrArgs& a) { return up(2 * (size_t)a.B * tiles_of(a) * a.D * sizeof(float)); }

}  // namespace

size_t glr_workspace_bytes(const GlrArgs& a, bool backward) {
    size_t scan = 0;
    for (int width = 32; width <= 64; width *= 2) {
        const size_t n = layout(a.B, a.T, a.D, width).bytes;
        scan = n > scan ? n : scan;
    }
    if (!backward) return scan;
    return scan + part_bytes(a) + up((size_t)a.B * tiles_of(a) * a.D * sizeof(float));
}

cudaError_t glr_bwd_read_and_clear_status(unsigned* value, bool clear) {
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return e;
    e = cudaMemcpyFromSymbol(value, g_glr_bwd_status, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_glr_bwd_status, &zero, sizeof(unsigned));
}

cudaError_t launch_glr_bwd(const GlrArgs& args, cudaStream_t s) {
    GlrArgs a = args;
    BwdSpace sp;
    char* ws = static_cast<char*>(a.ws);
    sp.scan = ws;
    ws += glr_workspace_bytes(a, false);
    sp.part = reinterpret_cast<float*>(ws);
    if (!a.ckpt) {
        a.ckpt = reinterpret_cast<float*>(ws + part_bytes(a));
        GlrArgs f = a;
        f.o = nullptr;
        f.hT = nullptr;
        f.ws = sp.scan;
        const cudaError_t e = launch_glr_fwd(f, s);
        if (e != cudaSuccess) return e;
    }
    if (!a.bf16) return bwd_wide<float, float>(a, sp, s);
    return a.g_bf16 ? bwd_wide<bf16, bf16>(a, sp, s) : bwd_wide<bf16, float>(a, sp, s);
}

}  // namespace gdn
