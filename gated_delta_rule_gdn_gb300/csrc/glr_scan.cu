// Gated linear recurrence: scan forward, and the decode step.
//   h_t = a_t h_{t-1} + u_t,  o_t = h_t;  see glr_math.cuh for a and u, glr_scan.cuh for the tiling and the carry.
// Bound by HBM: x, g and in_gate are read once and o is written once.

#include <type_traits>

#include "glr_scan.cuh"

namespace gdn {
namespace {

using namespace glr;
using mix::bf16;
using mix::Vec;

__device__ unsigned g_glr_status;   // bit 0: a block gave up a bounded wait

// one block per tile of 64 tokens x 32 V channels
template <typename Tx, typename Tg, int V>
__global__ void __launch_bounds__(kWarps * 32)
glr_fwd_kernel(const GlrArgs a, const Exchange x, int publish) {
    constexpr int W = 32 * V;
    __shared__ float sA[kWarps][W], sH[kWarps][W], s_carry[W];
    __shared__ int s_start[kTile], s_end[kTile];
    __shared__ unsigned s_id;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    unsigned id = blockIdx.x;
    if (x.tiles > 1) {
        if (tid == 0) s_id = atomicAdd(x.ticket, 1u);
        __syncthreads();
        id = s_id;
    }
    const int p = id / x.chains, chain = id % x.chains, cols = x.chains / a.B;
    const int b = chain / cols, c0 = (chain % cols) * W, c = c0 + lane * V;
    const int t0 = p * kTile + warp * kRun;
    const bool live = c < a.D;
    const size_t row0 = (size_t)b * a.T;

    // the run's inputs
    Vec<Tg, V> g[kRun];
    Vec<Tx, V> xv[kRun], gi[kRun];
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
        const bool in = live && t0 + j < a.T;
        if (in) g[j].load(static_cast<const Tg*>(a.g) + (row0 + t0 + j) * a.ldg + c); else g[j].zero();
        if (in) xv[j].load(static_cast<const Tx*>(a.x) + (row0 + t0 + j) * a.ldx + c); else xv[j].zero();
        if (a.gi) {
            if (in) gi[j].load(static_cast<const Tx*>(a.gi) + (row0 + t0 + j) * a.ldi + c); else gi[j].zero();
        }
    }
    // packed sequences: the one that starts at each token of the tile, and the one that ends there
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
    if (a.cu) __syncthreads();
    const unsigned starts = a.cu ? __ballot_sync(~0u, lane < kRun && s_start[warp * kRun + (lane & (kRun - 1))] >= 0) : 0;

    float al[kRun][V], u[kRun][V];
#pragma unroll
    for (int j = 0; j < kRun; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            al[j][v] = g[j].get(v);
            u[j][v] = xv[j].get(v);
        }
    if (a.A_log) {
        Channel ch[V];
#pragma unroll
        for (int v = 0; v < V; ++v) ch[v] = live ? channel(a.A_log, a.dt_bias, c + v) : Channel{0.f, 0.f};
#pragma unroll
        for (int j = 0; j < kRun; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) al[j][v] = ch[v].neg_eA * softplus(tail(al[j][v] + ch[v].dt));
    }
    if (a.gi) {
#pragma unroll
        for (int j = 0; j < kRun; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) u[j][v] *= sigmoid(tail(gi[j].get(v)));
    }
#pragma unroll
    for (int j = 0; j < kRun; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Decay d = decay(al[j][v]);
            if (a.normalize) u[j][v] *= input_factor(d);
            al[j][v] = t0 + j < a.T ? d.a : 1.f;         // past the row's end the state stays
        }

    // the run's map
    float A[V], H[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        A[v] = 1.f;
        H[v] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
        const bool starts_here = (starts >> j) & 1;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (starts_here) {
                const int n = s_start[warp * kRun + j];
                if (a.h0 && live) u[j][v] = fmaf(al[j][v], a.h0[(size_t)n * a.D + c + v], u[j][v]);
                H[v] = u[j][v];
            } else {
                H[v] = fmaf(al[j][v], H[v], u[j][v]);
                A[v] *= al[j][v];
            }
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        sA[warp][lane * V + v] = starts ? -1.f : A[v];
        sH[warp][lane * V + v] = H[v];
    }
    __syncthreads();

    // the tile's map, and the state that enters it
    float tA = 1.f, tH = 0.f, first = 0.f;
    if (tid < W) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            tH = apply(sA[w][tid], sH[w][tid], tH);
            tA = both(tA, sA[w][tid]);
        }
        if (p < kGroup && !a.cu && a.h0 && c0 + tid < a.D) first = a.h0[(size_t)b * a.D + c0 + tid];
    }
    const float carry = carry_in(x, W, p, chain, tA, tH, first, publish || p > 0, &g_glr_status);
    if (tid < W) {
        s_carry[tid] = carry;
        if (a.ckpt && c0 + tid < a.D && p * kTile < a.T)
            a.ckpt[((size_t)b * x.tiles + p) * a.D + c0 + tid] = carry;
    }
    __syncthreads();

    // the states
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = s_carry[lane * V + v];
    for (int w = 0; w < warp; ++w)
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = apply(sA[w][lane * V + v], sH[w][lane * V + v], h[v]);
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
        const bool starts_here = (starts >> j) & 1;
        Vec<Tx, V> o;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            h[v] = starts_here ? u[j][v] : fmaf(al[j][v], h[v], u[j][v]);
            o.set(v, h[v]);
        }
        if (a.o && live && t0 + j < a.T) o.store(static_cast<Tx*>(a.o) + (row0 + t0 + j) * a.D + c);
        if (a.cu && a.hT && live) {
            const int n = s_end[warp * kRun + j];
            if (n >= 0)
#pragma unroll
                for (int v = 0; v < V; ++v) a.hT[(size_t)n * a.D + c + v] = h[v];
        }
    }
    if (!a.hT || !live) return;
    if (!a.cu) {
        if (p == x.tiles - 1 && warp == kWarps - 1)
#pragma unroll
            for (int v = 0; v < V; ++v) a.hT[(size_t)b * a.D + c + v] = h[v];
    } else {
        // empty sequences end as they began; the row's tiles share them
        for (int n = p * kWarps + warp; n < a.n_seqs; n += x.tiles * kWarps) {
            if (mix::clamp_off(a.cu[n + 1], a.T) > mix::clamp_off(a.cu[n], a.T)) continue;
#pragma unroll
            for (int v = 0; v < V; ++v) a.hT[(size_t)n * a.D + c + v] = a.h0 ? a.h0[(size_t)n * a.D + c + v] : 0.f;
        }
    }
}

template <typename Tx, typename Tg>
__global__ void glr_step_kernel(const GlrStepArgs a) {
    const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t n = id / a.D;
    const int c = (int)(id % a.D);
    if (n >= a.N) return;
    const float g = mix::ld(static_cast<const Tg*>(a.g) + n * a.ldg + c);
    const Channel ch = channel(a.A_log, a.dt_bias, c);
    const Decay d = decay(a.A_log ? ch.neg_eA * softplus(tail(g + ch.dt)) : g);
    float u = mix::ld(static_cast<const Tx*>(a.x) + n * a.ldx + c);
    if (a.normalize) u *= input_factor(d);
    if (a.gi) u *= sigmoid(tail(mix::ld(static_cast<const Tx*>(a.gi) + n * a.ldi + c)));
    const float h = fmaf(d.a, a.h[n * a.D + c], u);
    a.h_out[n * a.D + c] = h;
    mix::st(static_cast<Tx*>(a.o) + n * a.D + c, h);
}

template <typename Tx, typename Tg, int V>
cudaError_t fwd(const GlrArgs& a, bool stall, cudaStream_t s) {
    const Layout l = layout(a.B, a.T, a.D, 32 * V);
    const Exchange x = exchange(l, a.ws);
    if (l.flag_bytes) {
        const cudaError_t e = cudaMemsetAsync(a.ws, 0, l.flag_bytes, s);
        if (e != cudaSuccess) return e;
    }
    glr_fwd_kernel<Tx, Tg, V><<<(unsigned)l.tiles * l.chains, kWarps * 32, 0, s>>>(a, x, stall ? 0 : 1);
    return cudaGetLastError();
}

template <typename Tx, typename Tg>
cudaError_t fwd_wide(const GlrArgs& a, bool stall, cudaStream_t s) {
    if (glr_vector(a, 4)) return fwd<Tx, Tg, 4>(a, stall, s);
    if (glr_vector(a, 2)) return fwd<Tx, Tg, 2>(a, stall, s);
    return fwd<Tx, Tg, 1>(a, stall, s);
}

}  // namespace

// Whether rows can be read and written V channels at a time.
bool glr_vector(const GlrArgs& a, int V) {
    const size_t es = a.bf16 ? 2 : 4, gs = a.g_bf16 ? 2 : 4;
    const auto ok = [V](const void* p, size_t size) { return reinterpret_cast<uintptr_t>(p) % (V * size) == 0; };
    return a.D % V == 0 && a.ldx % V == 0 && a.ldg % V == 0 && (!a.gi || a.ldi % V == 0) && ok(a.x, es) && ok(a.g, gs) &&
           ok(a.gi, es) && ok(a.o, es) && ok(a.dO, es) && ok(a.dx, es) && ok(a.dg, gs) && ok(a.di, es);
}

cudaError_t launch_glr_fwd(const GlrArgs& a, cudaStream_t s) {
    const bool stall = a.test_stall;
    if (!a.bf16) return fwd_wide<float, float>(a, stall, s);
    return a.g_bf16 ? fwd_wide<bf16, bf16>(a, stall, s) : fwd_wide<bf16, float>(a, stall, s);
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
