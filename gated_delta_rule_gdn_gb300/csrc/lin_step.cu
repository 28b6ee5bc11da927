// Decode step of linear attention with a decay for each head: h' = e^g h + k v^T, o = scale h'^T q, one token for each of N
// sequences.  Bound by the state, read and written once; the rest of a (sequence, head) is three vectors.
//
// A block takes some columns of one (sequence, head): all its threads hold V columns of every RG-th row between the read and
// the write, eight rows' reads in flight, and the rows' parts of o are joined in shared memory.  The columns of a head are
// spread over blocks of 32 where that many heads do not fill the card, else one block takes 128.
// (256 sequences of 32 heads of 128: 158 us, the copy rate; one sequence of 16: 4.1 us, the call.)

#include "lin_common.cuh"

namespace gdn {
namespace {

using mix::bf16;
constexpr int THREADS = 256, FLIGHT = 8;

template <typename T, int V, int LANES>                // LANES threads of V columns side by side
__global__ void __launch_bounds__(THREADS) lin_step_kernel(const LinStepArgs a) {
    constexpr int COLS = V * LANES, RG = THREADS / LANES;
    __shared__ float ks[256], qs[256];
    __shared__ float red[RG][COLS];
    const int tid = threadIdx.x, lane = tid % LANES, rg = tid / LANES;
    const int blocks = (a.dv + COLS - 1) / COLS;
    const int blk = blockIdx.x % blocks;
    const int64_t nh = blockIdx.x / blocks;
    const int h = (int)(nh % a.H);
    const int64_t n = nh / a.H;
    const int c0 = blk * COLS + lane * V;
    const bool in = c0 < a.dv;                         // (V divides dv)
    const float* src = a.state + nh * a.dk * a.dv + c0;
    float* dst = a.state_out + nh * a.dk * a.dv + c0;

    using S = mix::Vec<float, V>;
    S x[FLIGHT];
    auto read = [&](int r0) {
#pragma unroll
        for (int u = 0; u < FLIGHT; ++u) {
            const int r = r0 + u * RG;
            if (in && r < a.dk) {
                if constexpr (V == 4) {
                    const float4 f = __ldcs(reinterpret_cast<const float4*>(src + (int64_t)r * a.dv));
                    x[u].e[0] = f.x; x[u].e[1] = f.y; x[u].e[2] = f.z; x[u].e[3] = f.w;
                } else {
                    x[u].e[0] = __ldcs(src + (int64_t)r * a.dv);
                }
            }
        }
    };
    read(rg);
    const T* q = static_cast<const T*>(a.q.p) + n * a.q.tok + (h / a.q.group) * a.q.head;
    const T* k = static_cast<const T*>(a.k.p) + n * a.k.tok + (h / a.k.group) * a.k.head;
    const T* v = static_cast<const T*>(a.v.p) + n * a.v.tok + (h / a.v.group) * a.v.head;
    for (int i = tid; i < a.dk; i += THREADS) {
        ks[i] = mix::ld(k + i);
        qs[i] = mix::ld(q + i);
    }
    const float keep = expf(a.g[n * a.g_tok + h * a.g_head]);
    float vv[V], o[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        vv[i] = in ? mix::ld(v + c0 + i) : 0.f;
        o[i] = 0.f;
    }
    __syncthreads();
    for (int r0 = rg; r0 < a.dk; r0 += RG * FLIGHT) {
        if (r0 > rg) read(r0);
#pragma unroll
        for (int u = 0; u < FLIGHT; ++u) {
            const int r = r0 + u * RG;
            if (in && r < a.dk) {
                const float kr = ks[r], qr = qs[r];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    x[u].e[i] = fmaf(keep, x[u].e[i], kr * vv[i]);
                    o[i] = fmaf(qr, x[u].e[i], o[i]);
                }
                if constexpr (V == 4)
                    __stcs(reinterpret_cast<float4*>(dst + (int64_t)r * a.dv), make_float4(x[u].e[0], x[u].e[1], x[u].e[2], x[u].e[3]));
                else
                    __stcs(dst + (int64_t)r * a.dv, x[u].e[0]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) red[rg][lane * V + i] = o[i];
    __syncthreads();
    if (tid < COLS && blk * COLS + tid < a.dv) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < RG; ++i) s += red[i][tid];
        mix::st(static_cast<T*>(a.o) + nh * a.dv + blk * COLS + tid, a.scale * s);
    }
}

template <typename T, int V, int LANES>
cudaError_t start(const LinStepArgs& a, cudaStream_t s) {
    const int64_t blocks = (int64_t)a.N * a.H * ((a.dv + V * LANES - 1) / (V * LANES));
    lin_step_kernel<T, V, LANES><<<(unsigned)blocks, THREADS, 0, s>>>(a);
    return cudaGetLastError();
}
template <typename T>
cudaError_t typed(const LinStepArgs& a, cudaStream_t s) {
    const bool vec = a.dv % 4 == 0 && (uintptr_t)a.state % 16 == 0 && (uintptr_t)a.state_out % 16 == 0;
    if (!vec) return start<T, 1, 32>(a, s);
    return (int64_t)a.N * a.H >= 512 ? start<T, 4, 32>(a, s) : start<T, 4, 8>(a, s);
}

}  // namespace

cudaError_t launch_lin_step(const LinStepArgs& a, cudaStream_t s) { return a.bf16 ? typed<bf16>(a, s) : typed<float>(a, s); }

}  // namespace gdn
