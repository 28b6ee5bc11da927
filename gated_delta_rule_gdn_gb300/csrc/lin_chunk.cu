// Linear attention with a decay for each head on the tensor cores: the walk of lin.h for bf16 tokens, head sizes up to 128.
//
// One block walks one (sequence, value head, 64 columns of c) in chunks of 128 tokens.  With A, B [128, d] and C [128, 64] the
// tiles of a chunk, G the prefix sums of its log decays and S the fp32 state [d, 64]:
//     raw = A B^T                         P_ij = s_intra e^(G_i - G_j) raw_ij, j <= i (rev: e^(G_j - G_i), j >= i)
//     out = diag(s_inter e^G) A S + P C   S <- e^(G_end) S + B^T diag(s_state e^(G_end - G)) C
// Four products of 128 rows, so that each fills the 128 lanes of a tensor-core instruction; the state's own change does not
// depend on the state, so nothing but the fp32 update e^(G_end) S + dS is serial.
//
//   warps 0-3   scores: raw out of tensor memory, times decays, as bf16 back into tensor memory (the first operand of P C);
//               the outputs' epilogue
//   warps 4-7   state: in registers, a row a thread; scaled values and the state as operands in shared memory
//   warp 8      tensor copies: two stages of (A, B, C)
//   warp 9      issues the products
//   warp 10     prefix sums of the decays
//
// A block of 32 x 32 scores off the diagonal takes its decays as a product of two factors of at most one, e^(G_i - G_r) for
// the row and e^(G_r - G_j) for the column with r the row block's first (rev: last) token: one exponential for each of the
// block's columns in place of 32.  G is kept as the sum of two floats.
//
// Roundings: P and (without dots) the state as an operand go once to bf16, as the result does; scaled values always, and
// the state where an fp32 result comes of it, are the sum of two bf16 numbers (2^-18), in two products, the smaller first (the
// tensor cores' fp32 sums lose a little at every step, in proportion to the sum).
//
// A row of C that is not finite would reach the tokens before it as 0 times that; it is taken out of P C (not out of the
// state) and added to the rows that see it.

#include "internal.h"
#include "lin_common.cuh"
#include "tc_common.cuh"

namespace gdn {
namespace {

using namespace tc;
using mix::bf16;

__device__ unsigned g_lin_status;
__device__ __forceinline__ void report(unsigned bit) { atomicOr(&g_lin_status, bit); }

constexpr int CK = kLinChunk, NB = kLinCols;                    // tokens of a chunk, columns of c
constexpr uint64_t kWait = 2000000000ull;
constexpr int THREADS = 384;

// What a walk does besides: nothing, inner products of its rows with x (SPLIT: the state is exact enough for them), or the
// sums over pairs of tokens (PAIRS).
enum Kind { PLAIN, SPLIT, PAIRS };

struct Bars {
    uint64_t full[2], empty[2], raw_full, raw_free, ds_full, ds_free, s_ready, s_read, p_ready[2], o_full, o_free, vhat, gate_full,
        gate_empty, x_full, x_empty, sums_full, sums_read;
    uint32_t tmem;
    uint32_t flags[2][4];                                 // rows of C that are not finite, by chunk
};

template <Kind KIND>
struct Map {                                              // shared memory
    static constexpr uint32_t STAGE = 81920, A = 0, B = 32768, C = 65536;
    static constexpr uint32_t S = 2 * STAGE, V = S + (KIND == SPLIT ? 32768 : 16384), X = V + 32768;
    static constexpr uint32_t GH = X + (KIND == PAIRS ? 16384 : 0), GL = GH + 512, W = GL + 512, BARS = W + 1280;
    static constexpr uint32_t BYTES = BARS + sizeof(Bars);
    // tensor memory columns
    static constexpr uint32_t RAW = 0, P = 128, RAW2 = 192, DS = KIND == PAIRS ? 320 : 256, OI = KIND == PAIRS ? 384 : 320,
                              OA = KIND == PAIRS ? 448 : 384;
};
static_assert(Map<SPLIT>::BYTES <= 232448 && Map<PAIRS>::BYTES <= 232448, "shared memory of a block");
static_assert(Map<PAIRS>::OA + 64 <= 512, "tensor memory");

struct LinMaps { CUtensorMap a, b, c, x; };

__device__ __forceinline__ uint32_t bf2(float x, float y) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float finite_or_0(float x) { return fabsf(x) < INFINITY ? x : 0.f; }
// Column sums of a 32 x 32 block, a row a lane: lane l gets that of column l.
__device__ __forceinline__ float column_sums(float (&v)[32], int lane) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1)
#pragma unroll
        for (int k = 0; k < s; ++k) {
            const float send = lane & s ? v[k] : v[k + s], keep = lane & s ? v[k + s] : v[k];
            v[k] = keep + __shfl_xor_sync(0xffffffffu, send, s);
        }
    return v[0];
}

template <bool REV, Kind KIND>
__global__ void __launch_bounds__(THREADS, 1) lin_chunk_kernel(const __grid_constant__ LinMaps maps, const LinWalk w, float* pairs) {
    using M = Map<KIND>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    if (base & 1023u) {                                   // (the tiles' swizzle goes by address)
        if (threadIdx.x == 0) report(1u << 19);
        return;
    }
    Bars& S = *reinterpret_cast<Bars*>(smem + M::BARS);
    float* Gh = reinterpret_cast<float*>(smem + M::GH);
    float* Gl = reinterpret_cast<float*>(smem + M::GL);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int blocks = (w.dc + NB - 1) / NB;
    const int64_t unit = blockIdx.x;
    const int blk = (int)(unit % blocks), h = (int)(unit / blocks % w.H);
    const int n = lin::by_length(w.cu, w.n_seqs, w.T, (int)(unit / blocks / w.H));
    int64_t first;
    int len;
    lin::sequence(w.cu, w.T, n, first, len);
    const int chunks = (len + CK - 1) / CK;
    const int c0 = blk * NB, cols = min(NB, w.dc - c0);

    if (warp == 9) {
        tmem_alloc(&S.tmem, 512);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&S.full[s], 1);
            mbar_init(&S.empty[s], 1);
            mbar_init(&S.p_ready[s], 4);
        }
        mbar_init(&S.raw_full, 1);
        mbar_init(&S.raw_free, 4);
        mbar_init(&S.ds_full, 1);
        mbar_init(&S.ds_free, 4);
        mbar_init(&S.s_ready, 4);
        mbar_init(&S.s_read, 1);
        mbar_init(&S.o_full, 1);
        mbar_init(&S.o_free, 4);
        mbar_init(&S.vhat, 4);
        mbar_init(&S.gate_full, 1);
        mbar_init(&S.gate_empty, 8);
        mbar_init(&S.x_full, 1);
        mbar_init(&S.x_empty, 1);
        mbar_init(&S.sums_full, 4);
        mbar_init(&S.sums_read, 4);
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    bool ok = true;
    // chunk of a step, in the walk's direction, and how many of its tokens there are
    auto chunk_of = [&](int c) { return REV ? chunks - 1 - c : c; };
    auto rows_of = [&](int c) { return min(CK, len - chunk_of(c) * CK); };
    auto arrive = [&](uint64_t* bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    // (each wait for at most two seconds; all lanes of a warp give up together)
    auto wait = [&](uint64_t* bar, int phase, unsigned bit) {
        ok = mbar_wait(bar, phase & 1, kWait);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok && lane == 0) report(bit);
        return ok;
    };

    if (warp < 4) {
        // ------------------------------------------------------------------------------------- scores and outputs
        const int row = 32 * warp + lane;
        const uint32_t lanes = tmem + ((uint32_t)(32 * warp) << 16);
        // column factors of this warp's blocks off the diagonal, and with PAIRS its column sums: 32 floats a block
        constexpr int FIRST[2][4] = {{0, 32, 96, 192}, {0, 128, 224, 288}};
        float* W = reinterpret_cast<float*>(smem + M::W) + FIRST[REV ? 1 : 0][warp];
        const int J0 = REV ? warp : 0, J1 = REV ? 4 : warp + 1;
        float inter = 0.f;                                // s_inter e^(G_i), or e^(G_end - G_i), of the last two chunks
        float inter_before = 0.f;
        {   // the blocks on the other side of the diagonal stay zero
            uint32_t zero[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) zero[i] = 0u;
            for (int J = 0; J < 4; ++J)
                if (J < J0 || J >= J1) {
                    tmem_st16(lanes + M::P + 16 * J, zero);
                    if (KIND != PAIRS) tmem_st16(lanes + M::P + 64 + 16 * J, zero);
                }
            tmem_st_wait();
        }
        auto scores = [&](int c) {
            const int L = rows_of(c);
            const uint32_t p = lanes + M::P + (KIND == PAIRS ? 0 : (c & 1) * 64);
            if (!wait(&S.gate_full, c, 1u)) return;
            const float gh = Gh[row], gl = Gl[row];
            const int r = REV ? 32 * warp + 31 : 32 * warp;
            const float rh = Gh[r], rl = Gl[r], eh = Gh[CK - 1], el = Gl[CK - 1];
            inter_before = inter;
            inter = w.s_inter * (REV ? exp2f((eh - gh) + (el - gl)) : exp2f(gh + gl));
            const float u = w.s_intra * (REV ? exp2f((rh - gh) + (rl - gl)) : exp2f((gh - rh) + (gl - rl)));
            if (KIND == PAIRS && c > 0 && !wait(&S.sums_read, c - 1, 1u << 17)) return;
            for (int J = J0; J < J1; ++J)
                if (J != warp) {
                    const int j = 32 * J + lane;
                    W[32 * (J - J0) + lane] = REV ? exp2f((Gh[j] - rh) + (Gl[j] - rl)) : exp2f((rh - Gh[j]) + (rl - Gl[j]));
                }
            __syncwarp();
            if (!wait(&S.raw_full, c, 2u)) return;
            tc_fence_after();
            float sum = 0.f, other = 0.f;                 // over the pairs of row i (PAIRS): those off the diagonal
#pragma unroll 1
            for (int J = J0; J < J1; ++J) {
                uint32_t x[2][16], y[2][16];
                tmem_ld16(lanes + M::RAW + 32 * J, x[0]);
                tmem_ld16(lanes + M::RAW + 32 * J + 16, x[1]);
                if (KIND == PAIRS) {
                    tmem_ld16(lanes + M::RAW2 + 32 * J, y[0]);
                    tmem_ld16(lanes + M::RAW2 + 32 * J + 16, y[1]);
                }
                float f[32];
                if (J == warp) {
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 a = *reinterpret_cast<const float4*>(Gh + 32 * J + j);
                        const float4 b = *reinterpret_cast<const float4*>(Gl + 32 * J + j);
                        const float ah[4] = {a.x, a.y, a.z, a.w}, bl[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const bool in = REV ? j + i >= lane && 32 * J + j + i < L : j + i <= lane;
                            const float e = REV ? (ah[i] - gh) + (bl[i] - gl) : (gh - ah[i]) + (gl - bl[i]);
                            f[j + i] = in ? w.s_intra * exp2f(e) : 0.f;
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 a = *reinterpret_cast<const float4*>(W + 32 * (J - J0) + j);
                        f[j] = u * a.x;
                        f[j + 1] = u * a.y;
                        f[j + 2] = u * a.z;
                        f[j + 3] = u * a.w;
                    }
                }
                tmem_ld_wait();
                uint32_t q[16];
                // a score outside the triangle (or, rev, behind the sequence) is left out, not multiplied by nothing
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const bool in = (J != warp || (REV ? j >= lane : j <= lane)) && (!REV || 32 * J + j < L);
                    const float s = __uint_as_float(x[j >> 4][j & 15]) * f[j];
                    f[j] = in ? s : 0.f;
                }
#pragma unroll
                for (int j = 0; j < 32; j += 2) q[j >> 1] = bf2(f[j], f[j + 1]);
                tmem_st16(p + 16 * J, q);
                if (KIND == PAIRS) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const bool in = (J != warp || j != lane) && row < L && f[j] != 0.f;
                        f[j] = in ? f[j] * __uint_as_float(y[j >> 4][j & 15]) : 0.f;
                        sum += f[j];
                    }
                    const float s = column_sums(f, lane);
                    __syncwarp();
                    W[32 * (J - J0) + lane] = s;          // (the block's factors have been read)
                }
            }
            tc_fence_before();
            arrive(&S.gate_empty);
            arrive(&S.raw_free);
            tmem_st_wait();
            tc_fence_before();
            arrive(&S.p_ready[KIND == PAIRS ? 0 : c & 1]);
            if (KIND == PAIRS) {
                // row i of this walk is a key: its sum over the queries behind it; the sums over the keys before a query are
                // the column sums of the warps up to its own (the walk is a reverse one)
                arrive(&S.sums_full);
                if (!wait(&S.sums_full, c, 1u << 18)) return;
                const float* all = reinterpret_cast<const float*>(smem + M::W);
                for (int v = 0; v <= warp; ++v) other += all[FIRST[1][v] + 32 * (warp - v) + lane];
                if (row < L)
                    pairs[((int64_t)blk * w.H + h) * w.rows() + first + (int64_t)chunk_of(c) * CK + row] = other - sum;
                arrive(&S.sums_read);
            }
        };
        auto outputs = [&](int c, float f) {
            const int L = rows_of(c);
            const int64_t t = first + (int64_t)chunk_of(c) * CK + row;
            const bool in = row < L;
            uint4 xr[8];
            if (KIND == SPLIT) {
                const bf16* x = static_cast<const bf16*>(w.x.p) + t * w.x.tok + (h / w.x.group) * w.x.head + c0;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    xr[i] = in && 8 * i < cols ? *reinterpret_cast<const uint4*>(x + 8 * i) : make_uint4(0, 0, 0, 0);
            }
            if (!wait(&S.o_full, c, 4u)) return;
            tc_fence_after();
            uint32_t flags[4], any = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) any |= flags[i] = S.flags[c & 1][i];
            float o[64], dot = 0.f;
#pragma unroll
            for (int i = 0; i < 64; i += 16) {
                uint32_t a[16], b[16];
                tmem_ld16(lanes + M::OI + i, a);
                tmem_ld16(lanes + M::OA + i, b);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const float s = f * __uint_as_float(a[k]);
                    if (KIND == SPLIT) {
                        const uint4& v = xr[(i + k) >> 3];
                        const int e = (i + k) & 7;
                        const uint32_t word = e < 2 ? v.x : e < 4 ? v.y : e < 6 ? v.z : v.w;
                        dot = fmaf(e & 1 ? high(word) : low(word), s, dot);
                    }
                    o[i + k] = s + __uint_as_float(b[k]);
                }
            }
            if (any) {
                // rows of C that are not finite: into the rows that see them
                const bf16* cp = static_cast<const bf16*>(w.c.p) + (h / w.c.group) * w.c.head + c0;
                for (int j = 0; j < CK; ++j) {
                    if (!((flags[j >> 5] >> (j & 31)) & 1)) continue;
                    uint32_t pj[16];
                    tmem_ld16(lanes + M::P + (KIND == PAIRS ? 0 : (c & 1) * 64) + j / 32 * 16, pj);
                    tmem_ld_wait();
                    uint32_t word = 0;
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        if (k == (j & 31) / 2) word = pj[k];
                    const float p = j & 1 ? high(word) : low(word);
                    const bf16* cj = cp + (first + (int64_t)chunk_of(c) * CK + j) * w.c.tok;
                    if (REV ? row <= j : row >= j) {
#pragma unroll
                        for (int k = 0; k < 64; ++k)
                            if (k < cols) o[k] = fmaf(p, __bfloat162float(cj[k]), o[k]);
                    }
                }
            }
            tc_fence_before();
            arrive(&S.o_free);
            if (!in) return;
            if (KIND == SPLIT) w.dots[((int64_t)blk * w.H + h) * w.rows() + t] = dot;
            const int64_t at = (t * w.H + h) * w.dc + c0;
            if (w.out_f32) {
                float4* dst = reinterpret_cast<float4*>(static_cast<float*>(w.out) + at);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (4 * i < cols) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            } else {
                uint4* dst = reinterpret_cast<uint4*>(static_cast<bf16*>(w.out) + at);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (8 * i < cols)
                        dst[i] = make_uint4(bf2(o[8 * i], o[8 * i + 1]), bf2(o[8 * i + 2], o[8 * i + 3]),
                                            bf2(o[8 * i + 4], o[8 * i + 5]), bf2(o[8 * i + 6], o[8 * i + 7]));
            }
        };
        if (KIND == PAIRS) {                              // one buffer of P: its product first
            for (int c = 0; c < chunks && ok; ++c) {
                scores(c);
                if (ok) outputs(c, inter);
            }
        } else {                                          // the scores of the next chunk while this one's products run
            if (chunks > 0) scores(0);
            for (int c = 0; c < chunks && ok; ++c) {
                if (c + 1 < chunks) scores(c + 1);
                if (ok) outputs(c, c + 1 < chunks ? inter_before : inter);
            }
        }
    } else if (warp < 8) {
        // ------------------------------------------------------------------------------------------------- state
        const int row = tid - 128;                        // of the state, and of the chunk's tokens
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        float st[64];
        {
            const int64_t at = ((int64_t)n * w.H + h) * w.da * w.dc + (int64_t)row * w.s_r + (int64_t)c0 * w.s_c;
#pragma unroll
            for (int i = 0; i < 64; ++i) st[i] = w.s_in && row < w.da && i < cols ? w.s_in[at + (int64_t)i * w.s_c] : 0.f;
        }
        const int64_t slot0 = first / kLinSpan + n;
        // [span slot][h][block][row][column]
        auto span_at = [&](int ch) {
            return w.spans + ((((slot0 + ch / (kLinSpan / CK)) * w.H + h) * blocks + blk) * 128 + row) * (int64_t)NB;
        };
        auto operand = [&] {                              // S as an operand: rows of 64 columns, 128-byte swizzle
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float a = st[8 * i + 2 * k], b = st[8 * i + 2 * k + 1];
                    hi[k] = bf2(a, b);
                    if (KIND == SPLIT) lo[k] = bf2(finite_or_0(a - low(hi[k])), finite_or_0(b - high(hi[k])));
                }
                const uint32_t at = row * 128 + ((i ^ (row & 7)) << 4);
                sts128(base + M::S + at, hi[0], hi[1], hi[2], hi[3]);
                if (KIND == SPLIT) sts128(base + M::S + 16384 + at, lo[0], lo[1], lo[2], lo[3]);
            }
            fence_async_smem();
            arrive(&S.s_ready);
        };
        if (chunks > 0) operand();
        for (int c = 0; c < chunks; ++c) {
            const int s = c & 1, L = rows_of(c), ch = chunk_of(c);
            const uint32_t tile = base + s * M::STAGE;
            const bool starts_span = KIND == SPLIT && w.spans && ch % (kLinSpan / CK) == 0;
            if (starts_span && !REV) {                    // a span's first chunk: the state goes out
                float4* dst = reinterpret_cast<float4*>(span_at(ch));
#pragma unroll
                for (int i = 0; i < 16; ++i) dst[i] = make_float4(st[4 * i], st[4 * i + 1], st[4 * i + 2], st[4 * i + 3]);
            }
            if (!wait(&S.gate_full, c, 8u)) break;
            const float gh = Gh[row], gl = Gl[row], eh = Gh[CK - 1], el = Gl[CK - 1];
            arrive(&S.gate_empty);
            const float whole = exp2f(eh + el);
            if (starts_span && REV) {                     // or is multiplied with the one that did
                const float4* src = reinterpret_cast<const float4*>(span_at(ch));
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float4 x = src[i];
                    sum = fmaf(st[4 * i], x.x, sum);
                    sum = fmaf(st[4 * i + 1], x.y, sum);
                    sum = fmaf(st[4 * i + 2], x.z, sum);
                    sum = fmaf(st[4 * i + 3], x.w, sum);
                }
                for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
                if (lane == 0)
                    w.anchors[(((slot0 + ch / (kLinSpan / CK)) * w.H + h) * blocks + blk) * 4 + (warp & 3)] = whole * sum;
            }
            const float f = w.s_state * (REV ? exp2f(gh + gl) : exp2f((eh - gh) + (el - gl)));
            if (!wait(&S.full[s], c >> 1, 16u)) break;
            float nf = 0.f;                               // stays 0 unless an element is not finite
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t at = row * 128 + ((i ^ (row & 7)) << 4);
                const uint4 v = lds128(tile + M::C + at);
                const uint32_t word[4] = {v.x, v.y, v.z, v.w};
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float a = low(word[k]), b = high(word[k]);
                    if (row < L) nf = fmaf(a, 0.f, fmaf(b, 0.f, nf));
                    a = row < L ? f * a : 0.f;
                    b = row < L ? f * b : 0.f;
                    hi[k] = bf2(a, b);
                    lo[k] = bf2(a - low(hi[k]), b - high(hi[k]));
                }
                sts128(base + M::V + at, hi[0], hi[1], hi[2], hi[3]);
                sts128(base + M::V + 16384 + at, lo[0], lo[1], lo[2], lo[3]);
            }
            const bool odd = !(nf == 0.f);
            if (odd || row >= L) {                        // rare: a row to be passed over, or tokens of the next sequence (their
                                                          // scores, which may be under way, are left out in any case)
#pragma unroll
                for (int i = 0; i < 8; ++i) sts128(tile + M::C + row * 128 + i * 16, 0, 0, 0, 0);
                if (row >= L)
#pragma unroll
                    for (int i = 0; i < 16; ++i) sts128(tile + M::B + (i >> 3) * 16384 + row * 128 + (i & 7) * 16, 0, 0, 0, 0);
                if (odd)                                  // (the rest of an infinity is no number)
#pragma unroll 1
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t at = base + M::V + row * 128 + i * 16;
                        const uint4 lo = lds128(at + 16384);
                        const uint32_t word[4] = {lo.x, lo.y, lo.z, lo.w};
                        uint32_t z[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) z[k] = bf2(finite_or_0(low(word[k])), finite_or_0(high(word[k])));
                        sts128(at + 16384, z[0], z[1], z[2], z[3]);
                    }
            }
            const unsigned bits = __ballot_sync(0xffffffffu, odd && row < L);
            if (lane == 0) S.flags[c & 1][warp & 3] = bits;
            fence_async_smem();
            arrive(&S.vhat);
            if (!wait(&S.ds_full, c, 32u)) break;
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < 64; i += 32) {
                uint32_t a[2][16];
                tmem_ld16(lanes + M::DS + i, a[0]);
                tmem_ld16(lanes + M::DS + i + 16, a[1]);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 32; ++k) st[i + k] = fmaf(whole, st[i + k], __uint_as_float(a[k >> 4][k & 15]));
            }
            tc_fence_before();
            arrive(&S.ds_free);
            if (c + 1 < chunks) {
                if (!wait(&S.s_read, c, 64u)) break;
                operand();
            }
        }
        if (ok && w.s_out && row < w.da) {
            const int64_t at = ((int64_t)n * w.H + h) * w.da * w.dc + (int64_t)row * w.s_r + (int64_t)c0 * w.s_c;
#pragma unroll
            for (int i = 0; i < 64; ++i)
                if (i < cols) w.s_out[at + (int64_t)i * w.s_c] = st[i];
        }
    } else if (warp == 8) {
        // ------------------------------------------------------------------------------------------- tensor copies
        if (lane == 0 && chunks > 0) {
            prefetch_tmap(&maps.a);
            prefetch_tmap(&maps.b);
            prefetch_tmap(&maps.c);
            const int ha = h / w.a.group, hb = h / w.b.group, hc = h / w.c.group, hx = KIND == PAIRS ? h / w.x.group : 0;
            int issued = 0, issued_x = 0;
            uint64_t t_last = globaltimer_ns();
            while (issued < chunks || (KIND == PAIRS && issued_x < chunks)) {
                bool progress = false;
                if (issued < chunks) {
                    const int c = issued, s = c & 1;
                    if (c < 2 || mbar_test(&S.empty[s], ((c >> 1) + 1) & 1)) {
                        const int t = (int)(first + (int64_t)chunk_of(c) * CK);
                        uint8_t* tile = smem + s * M::STAGE;
                        mbar_arrive_expect_tx(&S.full[s], M::STAGE);
                        for (int i = 0; i < 2; ++i) {
                            tma_load_3d(tile + M::A + 16384 * i, &maps.a, &S.full[s], 64 * i, ha, t);
                            tma_load_3d(tile + M::B + 16384 * i, &maps.b, &S.full[s], 64 * i, hb, t);
                        }
                        tma_load_3d(tile + M::C, &maps.c, &S.full[s], c0, hc, t);
                        ++issued;
                        progress = true;
                    }
                }
                if (KIND == PAIRS && issued_x < chunks && (issued_x < 1 || mbar_test(&S.x_empty, (issued_x - 1) & 1))) {
                    const int t = (int)(first + (int64_t)chunk_of(issued_x) * CK);
                    mbar_arrive_expect_tx(&S.x_full, 16384);
                    tma_load_3d(smem + M::X, &maps.x, &S.x_full, c0, hx, t);
                    ++issued_x;
                    progress = true;
                }
                if (progress) t_last = globaltimer_ns();
                else if (globaltimer_ns() - t_last > kWait) {
                    report(128u);
                    break;
                }
            }
            // what was asked for has landed before the block leaves
            for (int c = issued > 2 ? issued - 2 : 0; c < issued; ++c) mbar_wait(&S.full[c & 1], (c >> 1) & 1, kWait);
            if (KIND == PAIRS && issued_x > 0) mbar_wait(&S.x_full, (issued_x - 1) & 1, kWait);
        }
    } else if (warp == 9) {
        // ------------------------------------------------------------------------------------------------ products
        if (lane == 0 && chunks > 0) {
            auto until = [&](uint64_t* bar, int phase, unsigned bit) {
                if (!ok) return false;
                ok = mbar_wait(bar, phase & 1, kWait);
                if (!ok) report(bit);
                return ok;
            };
            constexpr uint32_t id_raw = idesc_f16(128, 128, true, false, false);   // A (K-major) x B (K-major)
            constexpr uint32_t id_ds = idesc_f16(128, 64, true, true, true);       // B^T (MN-major) x scaled C (MN-major)
            constexpr uint32_t id_oi = idesc_f16(128, 64, true, false, true);      // A (K-major) x S (MN-major); P (TMEM) x C
            const int ksteps = (w.da + 15) / 16;
            auto scores = [&](int c) {
                const uint32_t tile = base + (c & 1) * M::STAGE;
                const uint64_t a = sdesc(tile + M::A, 16, 1024), b = sdesc(tile + M::B, 16, 1024);
                for (int k = 0; k < ksteps; ++k)
                    mma_f16(tmem + M::RAW, a + (k >> 2) * 1024 + (k & 3) * 2, b + (k >> 2) * 1024 + (k & 3) * 2, id_raw, k > 0);
                if (KIND != PAIRS) mma_commit(&S.raw_full);
            };
            if (until(&S.full[0], 0, 256u)) {
                tc_fence_after();
                if (KIND != PAIRS) scores(0);
            }
            for (int c = 0; c < chunks && ok; ++c) {
                const int s = c & 1;
                const uint32_t tile = base + s * M::STAGE;
                if (KIND == PAIRS) {
                    if (!until(&S.full[s], c >> 1, 256u) || (c > 0 && !until(&S.raw_free, c - 1, 512u))) break;
                    tc_fence_after();
                    scores(c);
                }
                if (!until(&S.vhat, c, 1u << 10) || (c > 0 && !until(&S.ds_free, c - 1, 1u << 11))) break;
                tc_fence_after();
                const uint64_t bt = sdesc(tile + M::B, 16384, 1024), v = sdesc(base + M::V, 16384, 1024);
#pragma unroll
                for (int k = 0; k < 8; ++k) mma_f16(tmem + M::DS, bt + k * 128, v + 1024 + k * 128, id_ds, k > 0);
#pragma unroll
                for (int k = 0; k < 8; ++k) mma_f16(tmem + M::DS, bt + k * 128, v + k * 128, id_ds, 1u);
                mma_commit(&S.ds_full);
                if (KIND == PAIRS) {                      // raw2 = X C^T (behind vhat: rows of C that are not finite are out)
                    if (!until(&S.x_full, c, 1u << 12)) break;
                    tc_fence_after();
                    const uint64_t x = sdesc(base + M::X, 16, 1024), ct = sdesc(tile + M::C, 16, 1024);
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_f16(tmem + M::RAW2, x + k * 2, ct + k * 2, id_raw, k > 0);
                    mma_commit(&S.raw_full);
                    mma_commit(&S.x_empty);
                } else if (c + 1 < chunks) {
                    if (!until(&S.full[s ^ 1], (c + 1) >> 1, 256u) || !until(&S.raw_free, c, 512u)) break;
                    tc_fence_after();
                    scores(c + 1);
                }
                if (!until(&S.s_ready, c, 1u << 13) || (c > 0 && !until(&S.o_free, c - 1, 1u << 14))) break;
                tc_fence_after();
                const uint64_t a = sdesc(tile + M::A, 16, 1024), so = sdesc(base + M::S, 16384, 1024);
                if (KIND == SPLIT)
                    for (int k = 0; k < ksteps; ++k)
                        mma_f16(tmem + M::OI, a + (k >> 2) * 1024 + (k & 3) * 2, so + 1024 + k * 128, id_oi, k > 0);
                for (int k = 0; k < ksteps; ++k)
                    mma_f16(tmem + M::OI, a + (k >> 2) * 1024 + (k & 3) * 2, so + k * 128, id_oi, KIND == SPLIT || k > 0);
                mma_commit(&S.s_read);
                if (!until(&S.p_ready[KIND == PAIRS ? 0 : s], KIND == PAIRS ? c : c >> 1, 1u << 15)) break;
                tc_fence_after();
                const uint64_t cm = sdesc(tile + M::C, 16384, 1024);
                const uint32_t p = tmem + M::P + (KIND == PAIRS ? 0 : s * 64);
#pragma unroll
                for (int k = 0; k < 8; ++k) mma_f16_ts(tmem + M::OA, p + 8 * k, cm + k * 128, id_oi, k > 0);
                mma_commit(&S.o_full);
                mma_commit(&S.empty[s]);
            }
        }
    } else if (warp == 10) {
        // ------------------------------------------------------------------------------------------------- decays
        auto fetch = [&](int c, float (&g)[4]) {
            const int L = c < chunks ? rows_of(c) : 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 4 * lane + i;
                g[i] = t < L ? w.g[(first + (int64_t)chunk_of(c) * CK + t) * w.g_tok + h * w.g_head] : 0.f;
            }
        };
        float g[4];
        fetch(0, g);
        for (int c = 0; c < chunks; ++c) {
            double s[4], sum = 0.0;
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] = sum += lin::log2_decay(g[i]);
            fetch(c + 1, g);
            double all = sum;
            for (int m = 1; m < 32; m <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, all, m);
                if (lane >= m) all += y;
            }
            if (c > 0 && !wait(&S.gate_empty, c - 1, 1u << 16)) break;
            float hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const double x = (all - sum) + s[i];
                hi[i] = (float)x;
                lo[i] = (float)(x - (double)hi[i]);
            }
            reinterpret_cast<float4*>(Gh)[lane] = make_float4(hi[0], hi[1], hi[2], hi[3]);
            reinterpret_cast<float4*>(Gl)[lane] = make_float4(lo[0], lo[1], lo[2], lo[3]);
            arrive(&S.gate_full);
        }
    }
    // every product has completed: the last chunk's are behind o_full (a walk that gave up waits as long as its waits)
    if (warp == 9 && lane == 0 && chunks > 0 && ok) mbar_wait(&S.o_full, (chunks - 1) & 1, kWait);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    __syncwarp();
    if (warp == 9) tmem_dealloc(tmem, 512);
}

// [tokens, heads, d] bf16 with strides: boxes of 64 channels x 1 head x 128 tokens
bool token_map(CUtensorMap* m, const LinTok& t, int d, int heads, int64_t rows) {
    return make_map_strided(m, t.p, rows, heads, d, t.tok, t.head, CK);
}

}  // namespace

bool lin_tensor_fits(const LinWalk& w) {
    auto fits = [](const LinTok& t) { return (uintptr_t)t.p % 16 == 0 && t.tok % 8 == 0 && t.head % 8 == 0; };
    return w.bf16 && w.da <= 128 && w.dc <= 128 && w.dc % 8 == 0 && fits(w.a) && fits(w.b) && fits(w.c) && (!w.x.p || fits(w.x)) &&
           (uintptr_t)w.out % 16 == 0 && device_is_sm100_family();
}

cudaError_t launch_lin_walk_tensor(const LinWalk& w, float* pairs, cudaStream_t s) {
    const int64_t units = (int64_t)w.N() * w.H * lin_blocks(w.dc, true);
    if (units == 0) return cudaSuccess;
    LinMaps maps{};
    const int64_t rows = w.rows() > 0 ? w.rows() : 1;
    if (w.rows() > 0) {
        if (!token_map(&maps.a, w.a, w.da, w.H / w.a.group, rows) || !token_map(&maps.b, w.b, w.da, w.H / w.b.group, rows) ||
            !token_map(&maps.c, w.c, w.dc, w.H / w.c.group, rows))
            return cudaErrorInvalidValue;
        if (pairs && !token_map(&maps.x, w.x, w.dc, w.H / w.x.group, rows)) return cudaErrorInvalidValue;
    }
    auto start = [&](auto kernel, uint32_t smem) -> cudaError_t {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        kernel<<<(unsigned)units, THREADS, smem, s>>>(maps, w, pairs);
        return cudaGetLastError();
    };
    if (pairs) return start(lin_chunk_kernel<true, PAIRS>, Map<PAIRS>::BYTES);
    if (w.dots) return w.rev ? start(lin_chunk_kernel<true, SPLIT>, Map<SPLIT>::BYTES) : start(lin_chunk_kernel<false, SPLIT>, Map<SPLIT>::BYTES);
    return start(lin_chunk_kernel<false, PLAIN>, Map<PLAIN>::BYTES);
}

cudaError_t lin_read_and_clear_status(unsigned* value, bool clear) {
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return e;
    e = cudaMemcpyFromSymbol(value, g_lin_status, sizeof(unsigned));
    if (e != cudaSuccess) return e;
    if (clear && *value) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_lin_status, &zero, sizeof(unsigned));
    }
    return e;
}

}  // namespace gdn
