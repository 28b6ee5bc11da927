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

template <typename Tx, typename Tg, int V>
__global__ void __launch_bounds__(kWarps * 32)
glr_bwd_kernel(const GlrArgs a, const Exchange x, float* part) {
    constexpr int W = 32 * V;
    __shared__ float sA[kWarps][W], sH[kWarps][W], sG[kWarps][W], s_carry[W], s_state[W];
    __shared__ int s_start[kTile], s_end[kTile];
    __shared__ unsigned s_id;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    unsigned id = blockIdx.x;
    if (x.tiles > 1) {
        if (tid == 0) s_id = atomicAdd(x.ticket, 1u);
        __syncthreads();
        id = s_id;
    }
    const int q = id / x.chains, p = x.tiles - 1 - q, chain = id % x.chains, cols = x.chains / a.B;
    const int b = chain / cols, c0 = (chain % cols) * W, c = c0 + lane * V;
    const int t0 = p * kTile + warp * kRun;
    const bool live = c < a.D;
    const size_t row0 = (size_t)b * a.T;

    Vec<Tg, V> g[kRun];
    Vec<Tx, V> xv[kRun], gi[kRun], dO[kRun];
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
        const bool in = live && t0 + j < a.T;
        if (in) g[j].load(static_cast<const Tg*>(a.g) + (row0 + t0 + j) * a.ldg + c); else g[j].zero();
        if (in) xv[j].load(static_cast<const Tx*>(a.x) + (row0 + t0 + j) * a.ldx + c); else xv[j].zero();
        if (in && a.gi) gi[j].load(static_cast<const Tx*>(a.gi) + (row0 + t0 + j) * a.ldi + c); else gi[j].zero();
        if (in) dO[j].load(static_cast<const Tx*>(a.dO) + (row0 + t0 + j) * a.D + c); else dO[j].zero();
    }
    if (a.cu && tid < kTile) {
        const int t = p * kTile + tid;
        int starts = -1, ends = -1;
        if (t < a.T) {
            const mix::Span s = mix::span_of(a.cu, a.n_seqs, a.T, t);
            if (s.first == t) starts = s.n;
            if (s.end == t + 1) ends = s.n;
        }
        s_start[tid] = starts;
        s_end[tid] = ends;
    }
    if (tid < W) {                               // the state that enters the tile
        float h = 0.f;
        if (c0 + tid < a.D && p * kTile < a.T) {
            if (p > 0 || a.cu) h = a.ckpt[((size_t)b * x.tiles + p) * a.D + c0 + tid];
            else if (a.h0) h = a.h0[(size_t)b * a.D + c0 + tid];
        }
        s_state[tid] = h;
    }
    __syncthreads();
    unsigned starts = 0, ends = 0;
    if (a.cu) {
        starts = __ballot_sync(~0u, lane < kRun && s_start[warp * kRun + (lane & (kRun - 1))] >= 0);
        ends = __ballot_sync(~0u, lane < kRun && s_end[warp * kRun + (lane & (kRun - 1))] >= 0);
    }
    Channel ch[V];
#pragma unroll
    for (int v = 0; v < V; ++v) ch[v] = live ? channel(a.A_log, a.dt_bias, c + v) : Channel{0.f, 0.f};

    // decays, the run's forward map (A, H) and backward map (A, G)
    float al[kRun][V], u[kRun][V];
#pragma unroll
    for (int j = 0; j < kRun; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float z = g[j].get(v);
            const Decay d = decay(a.A_log ? ch[v].neg_eA * softplus(tail(z + ch[v].dt)) : z);
            float w = xv[j].get(v);
            if (a.gi) w *= sigmoid(tail(gi[j].get(v)));
            if (a.normalize) w *= input_factor(d);
            u[j][v] = w;
            al[j][v] = t0 + j < a.T ? d.a : 1.f;
        }
    float A[V], H[V], G[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        A[v] = 1.f;
        H[v] = 0.f;
        G[v] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
        const bool here = (starts >> j) & 1;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (here) {
                const int n = s_start[warp * kRun + j];
                if (a.h0 && live) u[j][v] = fmaf(al[j][v], a.h0[(size_t)n * a.D + c + v], u[j][v]);
                H[v] = u[j][v];
            } else {
                H[v] = fmaf(al[j][v], H[v], u[j][v]);
            }
            A[v] *= al[j][v];
        }
    }
#pragma unroll
    for (int j = kRun - 1; j >= 0; --j) {
        const bool here = (ends >> j) & 1;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float D = dO[j].get(v);
            if (here) {
                const int n = s_end[warp * kRun + j];
                if (a.dhT && live) D += a.dhT[(size_t)n * a.D + c + v];
            } else {
                D += G[v];
            }
            G[v] = al[j][v] * D;
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        // one A serves both maps: the signs tell where each forgets
        sA[warp][lane * V + v] = A[v];
        sH[warp][lane * V + v] = H[v];
        sG[warp][lane * V + v] = G[v];
    }
    __shared__ unsigned char s_starts[kWarps], s_ends[kWarps];
    if (lane == 0) {
        s_starts[warp] = starts != 0;
        s_ends[warp] = ends != 0;
    }
    __syncthreads();
    float tA = 1.f, tG = 0.f, last = 0.f;
    if (tid < W) {
#pragma unroll
        for (int w = kWarps - 1; w >= 0; --w) {
            const float wA = s_ends[w] ? -1.f : sA[w][tid];
            tG = apply(wA, sG[w][tid], tG);
            tA = both(tA, wA);
        }
        if (q < kGroup && !a.cu && a.dhT && c0 + tid < a.D) last = a.dhT[(size_t)b * a.D + c0 + tid];
    }
    const float carry = carry_in(x, W, q, chain, tA, tG, last, true, &g_glr_bwd_status);
    if (tid < W) s_carry[tid] = carry;
    __syncthreads();

    // h_{t-1} of every token (in place of u), then the gradients from the last token to the first
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = s_state[lane * V + v];
    for (int w = 0; w < warp; ++w)
#pragma unroll
        for (int v = 0; v < V; ++v)
            h[v] = apply(s_starts[w] ? -1.f : sA[w][lane * V + v], sH[w][lane * V + v], h[v]);
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
        const bool here = (starts >> j) & 1;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float uj = u[j][v];
            if (here) {
                const int n = s_start[warp * kRun + j];
                u[j][v] = a.h0 && live ? a.h0[(size_t)n * a.D + c + v] : 0.f;
                h[v] = uj;
            } else {
                u[j][v] = h[v];
                h[v] = fmaf(al[j][v], h[v], uj);
            }
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) G[v] = s_carry[lane * V + v];
    for (int w = kWarps - 1; w > warp; --w)
#pragma unroll
        for (int v = 0; v < V; ++v)
            G[v] = apply(s_ends[w] ? -1.f : sA[w][lane * V + v], sG[w][lane * V + v], G[v]);
    float pA[V], pdt[V];
#pragma unroll
    for (int v = 0; v < V; ++v) pA[v] = pdt[v] = 0.f;
#pragma unroll
    for (int j = kRun - 1; j >= 0; --j) {
        const bool here = (ends >> j) & 1, in = live && t0 + j < a.T;
        Vec<Tx, V> dx, di;
        Vec<Tg, V> dg;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float D = dO[j].get(v);
            if (here) {
                const int n = s_end[warp * kRun + j];
                if (a.dhT && live) D += a.dhT[(size_t)n * a.D + c + v];
            } else {
                D += G[v];
            }
            G[v] = al[j][v] * D;
            const float z = g[j].get(v), xe = xv[j].get(v);
            const Tail tz = tail(z + ch[v].dt), ti = tail(gi[j].get(v));
            const float la = a.A_log ? ch[v].neg_eA * softplus(tz) : z;
            const float si = a.gi ? sigmoid(ti) : 1.f;
            float s = 1.f, dla = G[v] * u[j][v];
            if (a.normalize) {
                const Decay d = decay(la);
                s = input_factor(d);
                // ds/dlog a = -a^2 / s, taken as 0 where s = 0 (log a = 0: the derivative does not exist there)
                if (s > 0.f) dla -= D * si * xe * __fdividef(d.a * d.a, s);
            }
            const float du = D * s;
            dx.set(v, du * si);
            if (a.gi) di.set(v, du * xe * sigmoid_slope(ti));
            const float dz = a.A_log ? dla * ch[v].neg_eA * sigmoid(tz) : dla;
            dg.set(v, dz);
            if (in) {
                if (dla != 0.f) pA[v] = fmaf(dla, la, pA[v]);     // (0 where log a is infinite)
                pdt[v] += dz;
            }
        }
        if (in) {
            dx.store(static_cast<Tx*>(a.dx) + (row0 + t0 + j) * a.D + c);
            dg.store(static_cast<Tg*>(a.dg) + (row0 + t0 + j) * a.D + c);
            if (a.gi) di.store(static_cast<Tx*>(a.di) + (row0 + t0 + j) * a.D + c);
        }
        if (a.cu && a.dh0 && live) {
            const int n = s_start[warp * kRun + j];
            if (n >= 0)
#pragma unroll
                for (int v = 0; v < V; ++v) a.dh0[(size_t)n * a.D + c + v] = G[v];
        }
    }
    if (a.dh0 && live) {
        if (!a.cu) {
            if (p == 0 && warp == 0)
#pragma unroll
                for (int v = 0; v < V; ++v) a.dh0[(size_t)b * a.D + c + v] = G[v];
        } else {
            for (int n = p * kWarps + warp; n < a.n_seqs; n += x.tiles * kWarps) {
                if (mix::clamp_off(a.cu[n + 1], a.T) > mix::clamp_off(a.cu[n], a.T)) continue;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    a.dh0[(size_t)n * a.D + c + v] = a.dhT ? a.dhT[(size_t)n * a.D + c + v] : 0.f;
            }
        }
    }
    if (!a.dA) return;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) {
        sA[warp][lane * V + v] = pA[v];
        sG[warp][lane * V + v] = pdt[v];
    }
    __syncthreads();
    if (tid < W && c0 + tid < a.D) {
        float s = 0.f, d = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            s += sA[w][tid];
            d += sG[w][tid];
        }
        const size_t rows = (size_t)a.B * x.tiles, r = (size_t)b * x.tiles + p;
        part[r * a.D + c0 + tid] = s;
        part[(rows + r) * a.D + c0 + tid] = d;
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

template <typename Tx, typename Tg, int V>
cudaError_t bwd(const GlrArgs& a, const BwdSpace& sp, cudaStream_t s) {
    const Layout l = layout(a.B, a.T, a.D, 32 * V);
    const Exchange x = exchange(l, sp.scan);
    if (l.flag_bytes) {
        const cudaError_t e = cudaMemsetAsync(sp.scan, 0, l.flag_bytes, s);
        if (e != cudaSuccess) return e;
    }
    glr_bwd_kernel<Tx, Tg, V><<<(unsigned)l.tiles * l.chains, kWarps * 32, 0, s>>>(a, x, sp.part);
    if (a.dA)
        glr_param_kernel<<<dim3((a.D + 31) / 32, 2), 256, 0, s>>>(sp.part, a.B * l.tiles, a.D, a.dA, a.ddt);
    return cudaGetLastError();
}

template <typename Tx, typename Tg>
cudaError_t bwd_wide(const GlrArgs& a, const BwdSpace& sp, cudaStream_t s) {
    return glr_vector(a, 2) ? bwd<Tx, Tg, 2>(a, sp, s) : bwd<Tx, Tg, 1>(a, sp, s);
}

// The backward's workspace: the scan's exchange, the partial sums of the parameters, and the checkpoints that the
// caller did not keep (with the forward's exchange for computing them in the scan's place).
size_t up(size_t v) { return (v + 255) / 256 * 256; }
int tiles_of(const GlrArgs& a) { return layout(a.B, a.T, a.D, 32).tiles; }
size_t part_bytes(const GlrArgs& a) { return up(2 * (size_t)a.B * tiles_of(a) * a.D * sizeof(float)); }

}  // namespace

size_t glr_workspace_bytes(const GlrArgs& a, bool backward) {
    size_t scan = 0;
    for (int V = 1; V <= 4; V *= 2) {
        const size_t n = layout(a.B, a.T, a.D, 32 * V).bytes;
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
