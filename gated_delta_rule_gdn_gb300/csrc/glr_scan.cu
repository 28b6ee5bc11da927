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

template <typename Tx, typename Tg, int LANES, int V, bool PACKED>
__global__ void __launch_bounds__(kThreads, LANES * V <= 64 ? 3 : 2)
glr_fwd_kernel(const GlrArgs a, const Exchange x, const int publish) {
    using At = Place<LANES, V>;
    constexpr int W = At::W, R = At::kRuns, L = At::L;
    extern __shared__ __align__(16) unsigned char s_raw[];
    __shared__ float sA[R][W], sH[R][W];
    __shared__ int s_start[2][kTile], s_end[2][kTile];
    __shared__ unsigned s_next;
    const int tid = threadIdx.x, run = tid / LANES, lane = tid % LANES;
    auto* bg = reinterpret_cast<Vec<Tg, V>*>(s_raw) + tid;                    // [L][256] each
    auto* bx = reinterpret_cast<Vec<Tx, V>*>(s_raw + L * kThreads * sizeof(Vec<Tg, V>)) + tid;
    auto* bi = bx + L * kThreads;

    At at;
    const auto fetch = [&](int id) {
        at.set(x, a, id, false);
        const Tg* g = static_cast<const Tg*>(a.g) + at.row * a.ldg + at.c;
        const Tx* xp = static_cast<const Tx*>(a.x) + at.row * a.ldx + at.c;
        const Tx* ip = static_cast<const Tx*>(a.gi) + at.row * a.ldi + at.c;
        const int n = at.live ? at.count : 0;
#pragma unroll
        for (int j = 0; j < L; ++j) {
            mix::copy_async(bg + j * kThreads, j < n ? g : static_cast<const Tg*>(a.g), j < n);
            mix::copy_async(bx + j * kThreads, j < n ? xp : static_cast<const Tx*>(a.x), j < n);
            if (a.gi) mix::copy_async(bi + j * kThreads, j < n ? ip : static_cast<const Tx*>(a.gi), j < n);
            g += a.ldg;
            xp += a.ldx;
            ip += a.ldi;
        }
        mix::copies_close();
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
    if (id < x.total) {
        fetch(id);
        if (PACKED && tid < kTile) sequence_marks(a, at.p, s_start[0], s_end[0]);
    }
    if (PACKED) __syncthreads();

    for (int k = 0; id < x.total; k ^= 1) {
        const At now = at;
        // which tokens of the run start a sequence
        unsigned starts = 0;
        if (PACKED) {
#pragma unroll
            for (int j = 0; j < L; ++j) starts |= (s_start[k][run * L + j] >= 0 ? 1u : 0u) << j;
        }
        float al[L][V], u[L][V];
        mix::copies_wait<0>();
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
                const Vec<Tx, V> gi = bi[j * kThreads];
#pragma unroll
                for (int v = 0; v < V; ++v) u[j][v] *= sigmoid(gi.get(v));
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
                    const float z = al[j][v] + ch[v].dt;
                    al[j][v] = ch[v].neg_eA * softplus(z, tail(z));
                }
        } else {
#pragma unroll
            for (int j = 0; j < L; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) al[j][v] = min_nan(al[j][v], 88.f);
        }
#pragma unroll
        for (int j = 0; j < L; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Decay d = decay(al[j][v]);
                if (a.normalize) u[j][v] *= root(input_power(d));
                al[j][v] = d.a;
            }
        if (now.count < L) {                     // past the row's end the state stays
#pragma unroll
            for (int j = 0; j < L; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) al[j][v] = j < now.count ? al[j][v] : 1.f;
        }

        // the run's map
        float A[V], H[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            A[v] = al[0][v];
            H[v] = u[0][v];
        }
        if (PACKED && starts) {
#pragma unroll
            for (int j = 0; j < L; ++j) {
                const bool here = (starts >> j) & 1;
                if (here && a.h0 && now.live) {
                    const float* h0 = a.h0 + (size_t)s_start[k][run * L + j] * a.D + now.c;
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
            for (int j = 1; j < L; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    H[v] = fmaf(al[j][v], H[v], u[j][v]);
                    A[v] *= al[j][v];
                }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            sA[run][lane * V + v] = A[v];
            sH[run][lane * V + v] = H[v];
        }
        if (x.tiles > 1) {
            if (tid == 0) s_next = ticket;
        }
        __syncthreads();
        const int next = x.tiles > 1 ? (int)s_next : id + (int)gridDim.x;
        if (next < x.total) {                    // the buffer is free: the next tile's inputs on the way
            fetch(next);
            if (PACKED && tid < kTile) sequence_marks(a, at.p, s_start[k ^ 1], s_end[k ^ 1]);
            if (x.tiles > 1 && tid == 0) ticket = atomicAdd(x.ticket, 1u) + 1u;
        }

        // the state that enters the tile, and each of its runs
        if (tid < W) {
            const int c = now.c0 + tid;
            float tA = 1.f, tH = 0.f, h = 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                tH = apply(sA[r][tid], sH[r][tid], tH);
                tA = both(tA, sA[r][tid]);
            }
            if (!PACKED && now.p < kGroup && a.h0 && c < a.D) h = a.h0[(size_t)now.b * a.D + c];
            h = carry_in(x, W, now.p, now.chain, tid, tA, tH, h, publish || now.p > 0, &g_glr_status);
            if (a.ckpt && c < a.D && now.p * kTile < a.T) a.ckpt[((size_t)now.b * x.tiles + now.p) * a.D + c] = h;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float H = sH[r][tid];
                sH[r][tid] = h;
                h = apply(sA[r][tid], H, h);
            }
        }
        __syncthreads();

        float h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = sH[run][lane * V + v];
        Tx* op = static_cast<Tx*>(a.o) + now.row * a.D + now.c;
        const int n = now.live && a.o ? now.count : 0;
#pragma unroll
        for (int j = 0; j < L; ++j) {
            Vec<Tx, V> o;
            const bool here = PACKED && ((starts >> j) & 1);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                h[v] = here ? u[j][v] : fmaf(al[j][v], h[v], u[j][v]);
                o.set(v, h[v]);
            }
            if (j < n) o.store(op);
            op += a.D;
            if (PACKED && a.hT && now.live) {
                const int m = s_end[k][run * L + j];
                if (m >= 0)
#pragma unroll
                    for (int v = 0; v < V; ++v) a.hT[(size_t)m * a.D + now.c + v] = h[v];
            }
        }
        if (!PACKED && a.hT && now.live && now.p == x.tiles - 1 && run == R - 1)
#pragma unroll
            for (int v = 0; v < V; ++v) a.hT[(size_t)now.b * a.D + now.c + v] = h[v];
        if (PACKED && a.hT && now.live) {
            // empty sequences end as they began; the row's tiles share them
            for (int m = now.p * R + run; m < a.n_seqs; m += x.tiles * R) {
                if (mix::clamp_off(a.cu[m + 1], a.T) > mix::clamp_off(a.cu[m], a.T)) continue;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    a.hT[(size_t)m * a.D + now.c + v] = a.h0 ? a.h0[(size_t)m * a.D + now.c + v] : 0.f;
            }
        }
        id = next;
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
    float la = a.A_log ? ch.neg_eA * softplus(g + ch.dt, tail(g + ch.dt)) : min_nan(g, 88.f);
    const Decay d = decay(la);
    float u = mix::ld(static_cast<const Tx*>(a.x) + n * a.ldx + c);
    if (a.normalize) u *= root(input_power(d));
    if (a.gi) u *= sigmoid(mix::ld(static_cast<const Tx*>(a.gi) + n * a.ldi + c));
    const float h = fmaf(d.a, a.h[n * a.D + c], u);
    a.h_out[n * a.D + c] = h;
    mix::st(static_cast<Tx*>(a.o) + n * a.D + c, h);
}

template <typename Tx, typename Tg, int LANES, int V, bool PACKED>
cudaError_t fwd(const GlrArgs& a, cudaStream_t s) {
    using At = Place<LANES, V>;
    const Layout l = layout(a.B, a.T, a.D, At::W);
    const Exchange x = exchange(l, a.ws);
    if (l.bytes) {
        const cudaError_t e = cudaMemsetAsync(a.ws, 0xff, l.bytes, s);
        if (e != cudaSuccess) return e;
    }
    const auto kernel = glr_fwd_kernel<Tx, Tg, LANES, V, PACKED>;
    const size_t smem = (size_t)At::L * kThreads * V * (sizeof(Tg) + 2 * sizeof(Tx));
    static const Residency res = residency(reinterpret_cast<const void*>(kernel), smem);
    if (res.error != cudaSuccess) return res.error;
    kernel<<<x.total < res.blocks ? x.total : res.blocks, kThreads, smem, s>>>(a, x, a.test_stall ? 0 : 1);
    return cudaGetLastError();
}

template <typename Tx, typename Tg, int LANES, int V>
cudaError_t fwd_packed(const GlrArgs& a, cudaStream_t s) {
    return a.cu ? fwd<Tx, Tg, LANES, V, true>(a, s) : fwd<Tx, Tg, LANES, V, false>(a, s);
}

template <typename Tx, typename Tg>
cudaError_t fwd_wide(const GlrArgs& a, cudaStream_t s) {
    if (glr_vector(a, 4)) return fwd_packed<Tx, Tg, 16, 4>(a, s);
    if (glr_vector(a, 2)) return fwd_packed<Tx, Tg, 32, 2>(a, s);
    return fwd_packed<Tx, Tg, 32, 1>(a, s);
}

}  // namespace

// Blocks that are resident at once on the whole device (persistent kernels launch no more).
namespace glr {
Residency residency(const void* kernel, size_t smem) {
    Residency r{cudaSuccess, 0};
    int dev = 0, sms = 0, per = 0;
    r.error = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (r.error == cudaSuccess) r.error = cudaGetDevice(&dev);
    if (r.error == cudaSuccess) r.error = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (r.error == cudaSuccess) r.error = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, kThreads, smem);
    r.blocks = sms * (per > 0 ? per : 1);
    return r;
}
}  // namespace glr

// Whether rows can be read and written V channels at a time.
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
