// Gated linear recurrence: scan forward, its backward pass, and the decode step.
//   h_t = a_t h_{t-1} + u_t,  o_t = h_t;  see glr_math.cuh for a and u.
// Backward, with D_t the gradient of h_t: D_t = dO_t + a_{t+1} D_{t+1}, and the elementwise chain of each token.

#include <type_traits>

#include "glr_math.cuh"
#include "mixer.h"
#include "mixer_common.cuh"

namespace gdn {
namespace {

using mix::bf16;
using mix::ld;
using mix::st;

struct Channel { float neg_eA, dt; };   // -exp(A_log) (0: g is log a) and dt_bias of a channel
__device__ __forceinline__ Channel channel(const float* A_log, const float* dt_bias, int c) {
    return {A_log ? -expf(A_log[c]) : 0.f, dt_bias ? dt_bias[c] : 0.f};
}

struct Gate { float la, s; glr::Decay d; };
__device__ __forceinline__ Gate gate_of(bool act, bool norm, float g, const Channel& c) {
    Gate q;
    q.la = act ? c.neg_eA * glr::softplus(glr::tail(g + c.dt)) : g;
    q.d = glr::decay(q.la);
    q.s = norm ? glr::input_factor(q.d) : 1.f;
    return q;
}

// Gradients of one element: D the gradient of h_t, hp the state h_{t-1}, x the input, i its gate logit.  dla is the
// gradient of log a, dg that of g.  ds/dlog a = -a^2 / s is taken as 0 where s = 0 (log a = 0: it does not exist there).
struct Grad { float dx, dg, di, dla; };
__device__ __forceinline__ Grad grad_of(bool act, bool norm, bool gate, const Gate& q, float D, float hp, float x,
                                        float i, float g, const Channel& c) {
    Grad r;
    const glr::Tail ti = glr::tail(i);
    const float si = gate ? glr::sigmoid(ti) : 1.f, du = D * q.s;
    r.dx = du * si;
    r.di = du * x * glr::sigmoid_slope(ti);
    r.dla = q.d.a * D * hp;
    if (norm && q.s > 0.f) r.dla -= D * si * x * (q.d.a * q.d.a / q.s);
    r.dg = act ? r.dla * c.neg_eA * glr::sigmoid(glr::tail(g + c.dt)) : r.dla;
    return r;
}

// sequence n: its batch row and token range
__device__ __forceinline__ void sequence(const GlrArgs& a, int n, int* row, int* first, int* end) {
    *row = a.cu ? 0 : n;
    *first = a.cu ? mix::clamp_off(a.cu[n], a.T) : 0;
    *end = a.cu ? max(mix::clamp_off(a.cu[n + 1], a.T), *first) : a.T;
}

// one thread per (sequence, channel), token by token
template <typename Tx, typename Tg>
__global__ void glr_fwd_kernel(const GlrArgs a) {
    const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int n = (int)(id / a.D), c = (int)(id % a.D);
    if (n >= a.N()) return;
    int row, first, end;
    sequence(a, n, &row, &first, &end);
    const int tiles = (a.T + kGlrTile - 1) / kGlrTile;
    const Channel ch = channel(a.A_log, a.dt_bias, c);
    float h = a.h0 ? a.h0[(size_t)n * a.D + c] : 0.f;
    for (int t = first; t < end; ++t) {
        const size_t r = (size_t)row * a.T + t;
        if (a.ckpt && t % kGlrTile == 0) a.ckpt[((size_t)row * tiles + t / kGlrTile) * a.D + c] = h;
        const Gate q = gate_of(a.A_log, a.normalize, ld(static_cast<const Tg*>(a.g) + r * a.ldg + c), ch);
        float u = q.s * ld(static_cast<const Tx*>(a.x) + r * a.ldx + c);
        if (a.gi) u *= glr::sigmoid(glr::tail(ld(static_cast<const Tx*>(a.gi) + r * a.ldi + c)));
        h = fmaf(q.d.a, h, u);
        if (a.o) st(static_cast<Tx*>(a.o) + r * a.D + c, h);
    }
    if (a.hT) a.hT[(size_t)n * a.D + c] = h;
}

template <typename Tx, typename Tg>
__global__ void glr_bwd_kernel(const GlrArgs a, float* part) {
    const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int n = (int)(id / a.D), c = (int)(id % a.D);
    if (n >= a.N()) return;
    int row, first, end;
    sequence(a, n, &row, &first, &end);
    const int tiles = (a.T + kGlrTile - 1) / kGlrTile;
    const Channel ch = channel(a.A_log, a.dt_bias, c);
    const float h0 = a.h0 ? a.h0[(size_t)n * a.D + c] : 0.f;
    float G = a.dhT ? a.dhT[(size_t)n * a.D + c] : 0.f;   // gradient flowing into h_t from later tokens
    float sA = 0.f, sdt = 0.f;
    float hp[kGlrTile];
    for (int k = (end - 1) / kGlrTile; end > first && k >= first / kGlrTile; --k) {
        const int lo = max(first, k * kGlrTile), hi = min(end, (k + 1) * kGlrTile);
        float h = lo == first ? h0 : a.ckpt[((size_t)row * tiles + k) * a.D + c];
        for (int t = lo; t < hi; ++t) {
            const size_t r = (size_t)row * a.T + t;
            hp[t - k * kGlrTile] = h;
            const Gate q = gate_of(a.A_log, a.normalize, ld(static_cast<const Tg*>(a.g) + r * a.ldg + c), ch);
            float u = q.s * ld(static_cast<const Tx*>(a.x) + r * a.ldx + c);
            if (a.gi) u *= glr::sigmoid(glr::tail(ld(static_cast<const Tx*>(a.gi) + r * a.ldi + c)));
            h = fmaf(q.d.a, h, u);
        }
        for (int t = hi - 1; t >= lo; --t) {
            const size_t r = (size_t)row * a.T + t;
            const float g = ld(static_cast<const Tg*>(a.g) + r * a.ldg + c);
            const float x = ld(static_cast<const Tx*>(a.x) + r * a.ldx + c);
            const float i = a.gi ? ld(static_cast<const Tx*>(a.gi) + r * a.ldi + c) : 0.f;
            const Gate q = gate_of(a.A_log, a.normalize, g, ch);
            const float D = ld(static_cast<const Tx*>(a.dO) + r * a.D + c) + G;
            const Grad d = grad_of(a.A_log, a.normalize, a.gi, q, D, hp[t - k * kGlrTile], x, i, g, ch);
            G = q.d.a * D;
            st(static_cast<Tx*>(a.dx) + r * a.D + c, d.dx);
            st(static_cast<Tg*>(a.dg) + r * a.D + c, d.dg);
            if (a.gi) st(static_cast<Tx*>(a.di) + r * a.D + c, d.di);
            if (d.dla != 0.f) sA += d.dla * q.la;
            sdt += d.dg;
        }
    }
    if (a.dh0) a.dh0[(size_t)n * a.D + c] = G;
    if (a.dA) {
        part[(size_t)n * a.D + c] = sA;
        part[(size_t)(a.N() + n) * a.D + c] = sdt;
    }
}

__global__ void glr_param_kernel(const float* part, int N, int D, float* dA, float* ddt) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= D) return;
    float s = 0.f, u = 0.f;
    for (int n = 0; n < N; ++n) {
        s += part[(size_t)n * D + c];
        u += part[(size_t)(N + n) * D + c];
    }
    dA[c] = s;
    if (ddt) ddt[c] = u;
}

template <typename Tx, typename Tg>
__global__ void glr_step_kernel(const GlrStepArgs a) {
    const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t n = id / a.D;
    const int c = (int)(id % a.D);
    if (n >= a.N) return;
    const Gate q = gate_of(a.A_log, a.normalize, ld(static_cast<const Tg*>(a.g) + n * a.ldg + c),
                                channel(a.A_log, a.dt_bias, c));
    float u = q.s * ld(static_cast<const Tx*>(a.x) + n * a.ldx + c);
    if (a.gi) u *= glr::sigmoid(glr::tail(ld(static_cast<const Tx*>(a.gi) + n * a.ldi + c)));
    const float h = fmaf(q.d.a, a.h[n * a.D + c], u);
    a.h_out[n * a.D + c] = h;
    st(static_cast<Tx*>(a.o) + n * a.D + c, h);
}

template <typename F>
void by_type(bool x_bf16, bool g_bf16, F f) {
    if (!x_bf16) f((float*)nullptr, (float*)nullptr);
    else if (g_bf16) f((bf16*)nullptr, (bf16*)nullptr);
    else f((bf16*)nullptr, (float*)nullptr);
}

}  // namespace

size_t glr_workspace_bytes(const GlrArgs& a, bool backward) {
    if (!backward) return 0;
    const size_t tiles = (a.T + kGlrTile - 1) / kGlrTile;
    return ((size_t)a.B * tiles + 2 * (size_t)a.N()) * a.D * sizeof(float);
}

cudaError_t launch_glr_fwd(const GlrArgs& a, cudaStream_t s) {
    const unsigned blocks = (unsigned)(((int64_t)a.N() * a.D + 127) / 128);
    by_type(a.bf16, a.g_bf16, [&](auto* x, auto* g) {
        using Tx = std::remove_pointer_t<decltype(x)>;
        using Tg = std::remove_pointer_t<decltype(g)>;
        glr_fwd_kernel<Tx, Tg><<<blocks, 128, 0, s>>>(a);
    });
    return cudaGetLastError();
}

cudaError_t launch_glr_bwd(const GlrArgs& args, cudaStream_t s) {
    GlrArgs a = args;
    const unsigned blocks = (unsigned)(((int64_t)a.N() * a.D + 127) / 128);
    float* part = static_cast<float*>(a.ws);
    if (!a.ckpt) {
        a.ckpt = part + 2 * (size_t)a.N() * a.D;
        GlrArgs f = a;
        f.o = nullptr;
        f.hT = nullptr;
        const cudaError_t e = launch_glr_fwd(f, s);
        if (e != cudaSuccess) return e;
    }
    by_type(a.bf16, a.g_bf16, [&](auto* x, auto* g) {
        using Tx = std::remove_pointer_t<decltype(x)>;
        using Tg = std::remove_pointer_t<decltype(g)>;
        glr_bwd_kernel<Tx, Tg><<<blocks, 128, 0, s>>>(a, part);
    });
    if (a.dA) glr_param_kernel<<<(a.D + 127) / 128, 128, 0, s>>>(part, a.N(), a.D, a.dA, a.ddt);
    return cudaGetLastError();
}

cudaError_t launch_glr_step(const GlrStepArgs& a, cudaStream_t s) {
    const unsigned blocks = (unsigned)(((int64_t)a.N * a.D + 127) / 128);
    by_type(a.bf16, a.g_bf16, [&](auto* x, auto* g) {
        using Tx = std::remove_pointer_t<decltype(x)>;
        using Tg = std::remove_pointer_t<decltype(g)>;
        glr_step_kernel<Tx, Tg><<<blocks, 128, 0, s>>>(a);
    });
    return cudaGetLastError();
}

}  // namespace gdn
