// Linear attention with a decay for each head, backward: what the pairs of tokens of a chunk have of the decays' gradient.
//
// One block takes one chunk of 128 tokens of one head: Q K^T and dO V^T on the tensor cores, both in tensor memory, then
// M_ij = scale e^(G_i - G_j) (q_i . k_j) (dO_i . v_j) of the pairs j < i in fp32, summed along its rows (a row a lane) and its
// columns (over the lanes).  No chunk waits for another, so the bound is reading q, k, v and dO once; the two products share
// 64 KB of tiles one after the other, so that two blocks and more fit an SM and one loads while the others sum (4 sequences of 4096
// tokens, 16 heads of 128: 54 us, 40 at the copy rate; inside the walk of the values' gradient the sums took that from 71 to 180).

#include "lin_tile.cuh"

namespace gdn {
namespace {

__device__ unsigned g_lin_pairs_status;
__device__ __forceinline__ void report(unsigned bit) { atomicOr(&g_lin_pairs_status, bit); }

constexpr int THREADS = 160;                              // four warps that sum, one that loads and multiplies
struct PairBars {
    uint64_t full[2], done[2];
    uint32_t tmem;
};
constexpr uint32_t P_GH = 65536, P_GL = P_GH + 512, P_COLS = P_GL + 512, P_BARS = P_COLS + 2048, P_BYTES = P_BARS + sizeof(PairBars);
struct PairMaps { CUtensorMap q, k, o, v; };

__global__ void __launch_bounds__(THREADS, 2) lin_pairs_kernel(const __grid_constant__ PairMaps maps, const LinPairs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    mix::let_next();
    if (base & 1023u) {
        if (threadIdx.x == 0) report(1u);
        last_behind();
        return;
    }
    PairBars& S = *reinterpret_cast<PairBars*>(smem + P_BARS);
    float* Gh = reinterpret_cast<float*>(smem + P_GH);
    float* Gl = reinterpret_cast<float*>(smem + P_GL);
    float* cols = reinterpret_cast<float*>(smem + P_COLS);               // [row block][column]
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int h = blockIdx.x % a.H;
    const int64_t slot = blockIdx.x / a.H;
    const int n = lin::slot_sequence(a.cu, a.N(), a.T, CK, slot);
    int64_t first;
    int len;
    lin::sequence(a.cu, a.T, n, first, len);
    const int64_t at = (slot - (first / CK + n)) * CK;
    if (at < 0 || at >= len) {
        last_behind();
        return;
    }
    const int L = (int)min((int64_t)CK, len - at);
    const int64_t t0 = first + at;
    if (warp == 4) {
        tmem_alloc(&S.tmem, 256);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.full[i], 1);
            mbar_init(&S.done[i], 1);
        }
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, S.tmem, 0);
    bool ok = true;
    if (warp == 4) {
        constexpr uint32_t id = idesc_f16(128, 128, true, false, false);
        const uint64_t x = sdesc(base, 16, 1024), y = sdesc(base + 32768, 16, 1024);
        for (int i = 0; i < 2 && ok; ++i) {               // Q K^T, then dO V^T in its tiles' place
            if (elected()) {
                mbar_arrive_expect_tx(&S.full[i], 65536);
                for (int c = 0; c < 2; ++c) {
                    tma_load_3d(smem + 16384 * c, i ? &maps.o : &maps.q, &S.full[i], 64 * c, h / (i ? a.o.group : a.q.group), (int)t0);
                    tma_load_3d(smem + 32768 + 16384 * c, i ? &maps.v : &maps.k, &S.full[i], 64 * c, h / (i ? a.v.group : a.k.group), (int)t0);
                }
            }
            __syncwarp();
            ok = __all_sync(0xffffffffu, mbar_wait(&S.full[i], 0, kWait));
            if (!ok) {
                if (lane == 0) report(2u);
                break;
            }
            tc_fence_after();
            const bool wide = (i ? a.dv : a.dk) > 64;
            if (elected()) {
#pragma unroll
                for (int k = 0; k < 4; ++k) mma_f16(tmem + 128 * i, x + k * 2, y + k * 2, id, k > 0);
                if (wide)
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_f16(tmem + 128 * i, x + 1024 + k * 2, y + 1024 + k * 2, id, 1u);
                mma_commit(&S.done[i]);
            }
            __syncwarp();
            ok = __all_sync(0xffffffffu, mbar_wait(&S.done[i], 0, kWait));
            if (!ok && lane == 0) report(4u);
        }
    } else if (warp == 0) {                               // prefix sums of the decays
        lin::Log2 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 4 * lane + i;
            const lin::Log2 y = lin::log2_decay(t < L ? a.g[(t0 + t) * a.g_tok + h * a.g_head] : 0.f);
            x[i] = i > 0 ? lin::add(x[i - 1], y) : y;
        }
        const lin::Log2 all = lin::prefix(x[3], lane);
        const lin::Log2 before{__shfl_up_sync(0xffffffffu, all.hi, 1), __shfl_up_sync(0xffffffffu, all.lo, 1)};
        if (lane > 0)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = lin::add(before, x[i]);
        reinterpret_cast<float4*>(Gh)[lane] = make_float4(x[0].hi, x[1].hi, x[2].hi, x[3].hi);
        reinterpret_cast<float4*>(Gl)[lane] = make_float4(x[0].lo, x[1].lo, x[2].lo, x[3].lo);
    }
    __syncthreads();
    const int row = 32 * warp + lane;
    float sum = 0.f;
    if (warp < 4) {
        const uint32_t lanes = tmem + ((uint32_t)(32 * warp) << 16);
        const float gh = Gh[row], gl = Gl[row];
        ok = __all_sync(0xffffffffu, mbar_wait(&S.done[1], 0, kWait));
        if (!ok && lane == 0) report(8u);
        tc_fence_after();
#pragma unroll 1
        for (int J = 0; J <= warp; ++J) {
            uint32_t x[2][16], y[2][16];
            tmem_ld16(lanes + 32 * J, x[0]);
            tmem_ld16(lanes + 32 * J + 16, x[1]);
            tmem_ld16(lanes + 128 + 32 * J, y[0]);
            tmem_ld16(lanes + 128 + 32 * J + 16, y[1]);
            float m[32];
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const float4 p = *reinterpret_cast<const float4*>(Gh + 32 * J + j), r = *reinterpret_cast<const float4*>(Gl + 32 * J + j);
                m[j] = ex2((gh - p.x) + (gl - r.x));
                m[j + 1] = ex2((gh - p.y) + (gl - r.y));
                m[j + 2] = ex2((gh - p.z) + (gl - r.z));
                m[j + 3] = ex2((gh - p.w) + (gl - r.w));
            }
            tmem_ld_wait();
            // what is not a pair of this sequence is left out, not multiplied by nothing
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                const float v = m[j] * a.scale * __uint_as_float(x[j >> 4][j & 15]) * __uint_as_float(y[j >> 4][j & 15]);
                m[j] = row < L && (J != warp || j < lane) ? v : 0.f;
                sum += m[j];
            }
            cols[128 * warp + 32 * J + lane] = column_sums(m, lane);
        }
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (warp < 4 && row < L) {
        for (int i = warp; i < 4; ++i) sum -= cols[128 * i + row];
        a.pairs[(int64_t)h * a.rows() + t0 + row] = sum;
    }
    __syncwarp();
    if (warp == 4) tmem_dealloc(tmem, 256);
    last_behind();
}

}  // namespace

cudaError_t launch_lin_pairs(const LinPairs& a, cudaStream_t s) {
    if (a.rows() == 0) return cudaSuccess;
    PairMaps maps{};
    if (!token_map(&maps.q, a.q, a.dk, a.H / a.q.group, a.rows()) || !token_map(&maps.k, a.k, a.dk, a.H / a.k.group, a.rows()) ||
        !token_map(&maps.o, a.o, a.dv, a.H / a.o.group, a.rows()) || !token_map(&maps.v, a.v, a.dv, a.H / a.v.group, a.rows()))
        return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(lin_pairs_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)P_BYTES);
    if (e != cudaSuccess) return e;
    return mix::launch_behind(lin_pairs_kernel, dim3((unsigned)(lin_slots(a.rows(), a.N(), CK) * a.H)), THREADS, P_BYTES, true, s, maps, a);
}

cudaError_t lin_pairs_read_and_clear_status(unsigned* value, bool clear) {
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return e;
    e = cudaMemcpyFromSymbol(value, g_lin_pairs_status, sizeof(unsigned));
    if (e != cudaSuccess) return e;
    if (clear && *value) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_lin_pairs_status, &zero, sizeof(unsigned));
    }
    return e;
}

}  // namespace gdn
