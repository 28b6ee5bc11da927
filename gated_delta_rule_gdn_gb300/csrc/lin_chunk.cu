// Linear attention with a decay for each head on the tensor cores: the walk of lin.h for bf16 tokens, head sizes up to 128 (d_v of the forward up to 256).
//
// One block walks one (sequence, value head, 64 columns of c) in chunks of 128 tokens.  With A, B [128, d] and C [128, 64] the
// tiles of a chunk, G the prefix sums of its log decays and S the fp32 state [d, 64]:
//     raw = A B^T                         P_ij = s_intra e^(G_i - G_j) raw_ij, j <= i (rev: e^(G_j - G_i), j >= i)
//     out = diag(s_inter e^G) A S + P C   S <- e^(G_end) S + B^T diag(s_state e^(G_end - G)) C
// Four products of 128 rows, so that each fills the 128 lanes of a tensor-core instruction; the state's own change does not
// depend on the state, so nothing but the fp32 update e^(G_end) S + dS is serial.
//
// Where there are few sequences and heads, a walk is divided into segments: a first pass takes the state of each from nothing
// (STATE), a second joins them in order (lin_segments_kernel), and the walk proper starts each segment from its own state.
//
//   warps 0-7    scores and outputs, four warps a chunk in turn: raw out of tensor memory, times decays, as bf16 back into
//                tensor memory (the first operand of P C); the outputs' epilogue
//   warps 8-15   state, 32 columns a warpgroup: in registers, a row a thread; scaled values and the state as operands in
//                shared memory
//   warp 16      tensor copies: two stages of (A, B, C)
//   warp 17      issues the products
//   warp 18      decays: prefix sums, column factors
//
// The decays of a 32 x 32 block of scores off the diagonal are products of factors of at most one, e^(G_i - R_I) of the row (R the
// first token of its row block, E the last of a column block), e^(R_I - E_J) of the block and e^(E_J - G_j) of the column: one
// exponential for a column instead of 32 (rev: the other way round).  G is kept as the sum of two floats.
//
// Roundings: P and (without dots) the state as an operand go once to bf16, as the result does; scaled values always, and
// the state where an fp32 result comes of it, are the sum of two bf16 numbers (2^-17), in two products, the smaller first (the
// tensor cores' fp32 sums lose a little at every step, in proportion to the sum).  That leaves a state off by 4e-6 of its size.  In
// the walks behind the gradient of a constant decay (FINE), where the inner products of states enter for 128 tokens at once and
// their sum may be far below them, scaled values are three bf16 numbers, the third in the place of the state's operand once A S
// has read it: that gradient was off by up to 1.9e-5 of itself in 24 draws of B4, T 4096, 16 heads, and is by up to 3.6e-6; backward
// 356 -> 383 us there.  In the other walks it would cost more than it gives (forward 71 -> 99 us).
//
// A row of C that is not finite would reach the tokens before it as 0 times that; it is taken out of P C (not out of the
// state) and added to the rows that see it.
//
// What bounds it: no unit alone.  A chunk's operands and what is turned on the way are 336 KB of reads and writes of shared memory (SPLIT
// 464, FINE 528), so 1.3, 1.8 and 2.1 us at 128 bytes a cycle, of the 2.2, 3.9 and 4.4 that it takes; tensor pipe 38, 25 and 26 %, issue 44,
// 41 and 40 %, DRAM 43, 44 and 39 %.  The rest is what the roles wait for one another; it has not been taken apart.  128 walks fill 128 of
// 152 SMs.  B4, T 4096, 16 heads of 128: forward 71 us (58 % of the copy rate), dq 122, dk 130, dv 73 (FINE: dq 139, dk 145).  Not kept:
// four warps a role instead
// of eight (137 us forward), products from a branch of one lane instead of an elected one (70 to 150 cycles each, not 33 to 64), decays
// in 64 bits, the spans' states asked for a chunk ahead (backward of 65,536 tokens, 32 heads: 2.63 ms, 2.53 without).
//
// The kernels of a call are launched before the one before them has completed, and wait only where they read what it wrote: the walk
// of dv runs beside that of dk, the sums of pairs beside both, on the SMs that they leave (backward of B4, T 4096, 8 heads: 332 us one
// after another, 253 so; of 1000 tokens, 16 heads: 114 and 82; B4, T 4096, 16 heads: 390 and 352, with a constant decay 411 and 380).

#include <cmath>

#include "lin_tile.cuh"

namespace gdn {
namespace {

__device__ unsigned g_lin_status;
__device__ __forceinline__ void report(unsigned bit) { atomicOr(&g_lin_status, bit); }

constexpr int NB = kLinCols;                              // columns of c
constexpr int THREADS = 640;

// A walk; one that also takes inner products of its rows with x, for which the state as an operand is exact enough (SPLIT); or
// the state alone (STATE), of a segment from nothing.
enum Kind { PLAIN, SPLIT, STATE };
// s_ready, s_read: the state's operand is written, and read by A S; vhat, third: the scaled values are

struct Bars {
    uint64_t full[2], full_c[2], empty[2], empty_c[2], gate_empty[2], raw_full[2], p_ready[2], o_full[2], o_free[2];
    uint64_t ds_full, ds_free, s_ready, s_read, vhat, third;
    // Rows of C that are not finite, by chunk, half of the columns and 32 rows.  Four chunks' places: those of chunk c + 4 are
    // written behind ds_full of c + 2, whose product is issued behind the scores of c + 2 and so behind o_free of c, which the
    // score warps signal when they have read theirs for the last time.  (Two places would not do: without SPLIT nothing holds the
    // state warps back until the outputs of the chunk before last are done, and those take long beside such a row.)
    uint32_t flags[4][2][4];
    lin::Keep keep[2];                                    // of a chunk's whole decay
    uint32_t tmem;
};

template <Kind KIND>
struct Map {                                              // shared memory
    static constexpr uint32_t STAGE = 81920, A = 0, B = 32768, C = 65536;
    static constexpr uint32_t S = 2 * STAGE, V = S + (KIND == SPLIT ? 32768 : 16384), TURN = V + 32768;      // (where outputs turn)
    // two buffers of each: G rounded, what the rounding left (bf16), column factors
    static constexpr uint32_t GH = TURN + (KIND == PLAIN ? 16384 : 0), CF = GH + 1024, GL = CF + 1024, BARS = GL + 512;
    static constexpr uint32_t BYTES = BARS + sizeof(Bars);
    // Tensor memory columns: two buffers of scores, P in the first half of its scores and P C in the second; the two parts of
    // the state's change side by side; two buffers of A S.
    static constexpr uint32_t RAW = 0, P = 0, OA = 64, RING = 128, DS = 256, OI = 384, OI_RING = 64;
};
static_assert(Map<SPLIT>::BYTES <= 232448 && Map<PLAIN>::BYTES <= 232448, "shared memory of a block");

struct LinMaps { CUtensorMap a, b, c; };

// the larger magnitude of each half (and a sign of no meaning), NaN if either is
__device__ __forceinline__ uint32_t most(uint32_t a, uint32_t w) {
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t mul_bf(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t fma_bf(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
template <bool REV, Kind KIND, bool FINE>
__global__ void __launch_bounds__(THREADS, 1) lin_chunk_kernel(const __grid_constant__ LinMaps maps, const LinWalk w) {
    using M = Map<KIND>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    mix::let_next();
    if (base & 1023u) {                                   // (the tiles' swizzle goes by address)
        if (threadIdx.x == 0) report(1u << 19);
        last_behind();
        return;
    }
    Bars& S = *reinterpret_cast<Bars*>(smem + M::BARS);
    auto Gh = [&](int c) { return reinterpret_cast<float*>(smem + M::GH) + (c & 1) * CK; };
    auto Gl = [&](int c) { return reinterpret_cast<bf16*>(smem + M::GL) + (c & 1) * CK; };
    auto Cf = [&](int c) { return reinterpret_cast<float*>(smem + M::CF) + (c & 1) * CK; };

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int blocks = (w.dc + NB - 1) / NB;
    const int64_t unit = blockIdx.x;
    const int blk = (int)(unit % blocks), h = (int)(unit / blocks % w.H);
    const int64_t slot = unit / blocks / w.H;             // a sequence, or a segment of one
    int n = 0, len, base_chunk = 0, count;
    bool last = true;                                     // in the walk's direction
    int64_t first;
    if (w.seg_chunks > 0) {
        n = lin::slot_sequence(w.cu, w.N(), w.T, w.seg_chunks * CK, slot);
        lin::sequence(w.cu, w.T, n, first, len);
        const int64_t at = (slot - (first / (w.seg_chunks * CK) + n)) * w.seg_chunks;
        if (at < 0 || at * CK >= len) {                   // (a slot of no segment)
            last_behind();
            return;
        }
        base_chunk = (int)at;
        count = min(w.seg_chunks, (len + CK - 1) / CK - base_chunk);
        last = REV ? base_chunk == 0 : base_chunk + count == (len + CK - 1) / CK;
        if (KIND == STATE && last) {                      // (no segment enters behind it)
            last_behind();
            return;
        }
    } else {
        n = lin::by_length(w.cu, w.n_seqs, w.T, (int)slot);
        lin::sequence(w.cu, w.T, n, first, len);
        count = (len + CK - 1) / CK;
    }
    const int chunks = __shfl_sync(0xffffffffu, count, 0);
    const int c0 = blk * NB, cols = min(NB, w.dc - c0);

    if (warp == 17) {
        tmem_alloc(&S.tmem, 512);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&S.full[s], 2);                     // A and B, and the decays
            mbar_init(&S.full_c[s], 1);
            mbar_init(&S.empty[s], 1);
            mbar_init(&S.empty_c[s], KIND == SPLIT ? 4 : 1);
            mbar_init(&S.gate_empty[s], KIND == STATE ? 8 : 12);
            mbar_init(&S.raw_full[s], 1);
            mbar_init(&S.p_ready[s], 4);
            mbar_init(&S.o_full[s], 1);
            mbar_init(&S.o_free[s], 4);
        }
        mbar_init(&S.ds_full, 1);
        mbar_init(&S.ds_free, 8);
        mbar_init(&S.s_ready, 8);
        mbar_init(&S.s_read, 1);
        mbar_init(&S.vhat, 8);
        mbar_init(&S.third, 8);
        fence_mbar_init();
    }
    if (w.wait_first) mix::wait_behind();                 // (before any wait that is counted)
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, S.tmem, 0);
    bool ok = true;
    // chunk of a step, in the walk's direction, and how many of its tokens there are
    auto chunk_of = [&](int c) { return base_chunk + (REV ? chunks - 1 - c : c); };
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

    if (warp < 8 && KIND == STATE) {
        // (nothing to score)
    } else if (warp < 8) {
        // ------------------------------------------------------------------------------------- scores and outputs
        const int I = warp & 3, row = 32 * I + lane;
        const uint32_t lanes = tmem + ((uint32_t)(32 * I) << 16);
        const int J0 = REV ? I : 0, J1 = REV ? 4 : I + 1;
        const bf16* xp = static_cast<const bf16*>(w.x.p) + (h / w.x.group) * w.x.head + c0;
        for (int c = warp >> 2; c < chunks; c += 2) {
            const int L = rows_of(c), s = c & 1;
            const int64_t t0 = (int64_t)chunk_of(c) * CK;
            const uint32_t raw = lanes + M::RAW + s * M::RING, p = lanes + M::P + s * M::RING;
            if (!wait(&S.full[s], c >> 1, 1u)) break;
            const float *gh = Gh(c), *cf = Cf(c);
            const bf16* gl = Gl(c);
            const float ih = gh[row], il = __bfloat162float(gl[row]);
            const int r = 32 * I + (REV ? 31 : 0);
            const float rh = gh[r], rl = __bfloat162float(gl[r]);
            const float f_inter = w.s_inter * (REV ? ex2((gh[CK - 1] - ih) + (__bfloat162float(gl[CK - 1]) - il)) : ex2(ih + il));
            const float u = w.s_intra * (REV ? ex2((rh - ih) + (rl - il)) : ex2((ih - rh) + (il - rl)));
            if (!wait(&S.raw_full[s], c >> 1, 2u)) break;
            tc_fence_after();
#pragma unroll 1
            for (int J = J0; J < J1; ++J) {
                uint32_t xr[2][16];
                tmem_ld16(raw + 32 * J, xr[0]);
                tmem_ld16(raw + 32 * J + 16, xr[1]);
                float x[32];
                if (J == I) {
                    // on the diagonal an exponential each; what is outside the triangle is left out, not multiplied by nothing
                    float f[32];
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 a = *reinterpret_cast<const float4*>(gh + 32 * J + j);
                        const uint2 b = *reinterpret_cast<const uint2*>(gl + 32 * J + j);
                        const F2 h0{a.x, a.y}, h1{a.z, a.w}, l0{low(b.x), high(b.x)}, l1{low(b.y), high(b.y)}, m1{-1.f, -1.f};
                        const F2 e0 = REV ? add2(add2(h0, F2{-ih, -ih}), add2(l0, F2{-il, -il})) : add2(fma2(h0, m1, F2{ih, ih}), fma2(l0, m1, F2{il, il}));
                        const F2 e1 = REV ? add2(add2(h1, F2{-ih, -ih}), add2(l1, F2{-il, -il})) : add2(fma2(h1, m1, F2{ih, ih}), fma2(l1, m1, F2{il, il}));
                        f[j] = ex2(e0.x);
                        f[j + 1] = ex2(e0.y);
                        f[j + 2] = ex2(e1.x);
                        f[j + 3] = ex2(e1.y);
                    }
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const F2 v = mul2(mul2(F2{f[j], f[j + 1]}, F2{w.s_intra, w.s_intra}),
                                          F2{__uint_as_float(xr[j >> 4][j & 15]), __uint_as_float(xr[j >> 4][(j & 15) + 1])});
                        x[j] = (REV ? j >= lane : j <= lane) ? v.x : 0.f;
                        x[j + 1] = (REV ? j + 1 >= lane : j + 1 <= lane) ? v.y : 0.f;
                    }
                } else {
                    const int e = REV ? 32 * J : 32 * J + 31;
                    const float f = u * (REV ? ex2((gh[e] - rh) + (__bfloat162float(gl[e]) - rl)) : ex2((rh - gh[e]) + (rl - __bfloat162float(gl[e]))));
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 a = *reinterpret_cast<const float4*>(cf + 32 * J + j);
                        const F2 v0 = mul2(mul2(F2{a.x, a.y}, F2{f, f}), F2{__uint_as_float(xr[j >> 4][j & 15]), __uint_as_float(xr[j >> 4][(j & 15) + 1])});
                        const F2 v1 = mul2(mul2(F2{a.z, a.w}, F2{f, f}), F2{__uint_as_float(xr[j >> 4][(j & 15) + 2]), __uint_as_float(xr[j >> 4][(j & 15) + 3])});
                        x[j] = v0.x;
                        x[j + 1] = v0.y;
                        x[j + 2] = v1.x;
                        x[j + 3] = v1.y;
                    }
                }
                if (REV && L < CK)                        // tokens behind the sequence
#pragma unroll
                    for (int j = 0; j < 32; ++j) x[j] = 32 * J + j < L ? x[j] : 0.f;
                uint32_t q[16];
#pragma unroll
                for (int j = 0; j < 32; j += 2) q[j >> 1] = bf2(x[j], x[j + 1]);
                tmem_st16(p + 16 * J, q);
            }
            {   // the blocks on the other side of the diagonal
                uint32_t zero[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) zero[i] = 0u;
                for (int J = REV ? 0 : J1; J < (REV ? J0 : 4); ++J) tmem_st16(p + 16 * J, zero);
            }
            tc_fence_before();
            arrive(&S.gate_empty[s]);
            tmem_st_wait();
            tc_fence_before();
            arrive(&S.p_ready[s]);
            const bool in = row < L;
            const int64_t t = first + t0 + row;

            // rows of the outputs go, and rows of x come, several lanes a row (a lane a row would touch 32 lines an access):
            // turned in shared memory of the warp's own, 32 rows of 64 bytes, or in the chunk's C tile, which has been read
            // when the outputs are there, of 128
            constexpr int Q = KIND == PLAIN ? 4 : 8, RPA = 32 / Q;                // pieces of a row, rows of an access
            const uint32_t turn = KIND == PLAIN ? base + M::TURN + warp * 2048 : base + s * M::STAGE + M::C + I * 4096;
            const int rq = lane / Q, q = lane % Q;
            auto at_row = [&](int r, int i) { return turn + r * (16 * Q) + ((i ^ (KIND == PLAIN ? (r >> 1) & 3 : r & 7)) << 4); };
            uint4 xv[8];
            if (KIND == SPLIT)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = RPA * i + rq;
                    xv[i] = 32 * I + r < L && 8 * q < cols
                                ? *reinterpret_cast<const uint4*>(xp + (first + t0 + 32 * I + r) * w.x.tok + 8 * q)
                                : make_uint4(0, 0, 0, 0);
                }
            if (!wait(&S.o_full[s], c >> 1, 8u)) break;
            tc_fence_after();
            if (KIND == SPLIT) {
#pragma unroll
                for (int i = 0; i < 8; ++i) sts128(at_row(RPA * i + rq, q), xv[i].x, xv[i].y, xv[i].z, xv[i].w);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) xv[i] = lds128(at_row(lane, i));
                __syncwarp();
            }
            uint32_t any = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) any |= S.flags[c & 3][i >> 2][i & 3];
            F2 dot{0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 64; i += 16) {
                uint32_t a[16], b[16];
                tmem_ld16(lanes + M::OI + s * M::OI_RING + i, a);
                tmem_ld16(lanes + M::OA + s * M::RING + i, b);
                tmem_ld_wait();
                float o[16];
#pragma unroll
                for (int k = 0; k < 16; k += 2) {
                    const F2 g{__uint_as_float(a[k]), __uint_as_float(a[k + 1])};
                    if (KIND == SPLIT) {
                        const uint4& v = xv[(i + k) >> 3];
                        const int e = (k & 7) >> 1;
                        const uint32_t word = e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w;
                        dot = fma2(F2{low(word), high(word)}, g, dot);
                    }
                    const F2 v = fma2(F2{f_inter, f_inter}, g, F2{__uint_as_float(b[k]), __uint_as_float(b[k + 1])});
                    o[k] = v.x;
                    o[k + 1] = v.y;
                }
                if (any)                                  // rows of C that are not finite: into the rows that see them
#pragma unroll 1
                    for (int j = 0; j < CK; ++j) {
                        if (!((S.flags[c & 3][i >> 5][j >> 5] >> (j & 31)) & 1)) continue;
                        uint32_t pj[16];
                        tmem_ld16(p + j / 32 * 16, pj);
                        tmem_ld_wait();
                        uint32_t word = 0;
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            if (k == (j & 31) / 2) word = pj[k];
                        const float pv = j & 1 ? high(word) : low(word);
                        const bf16* cj = static_cast<const bf16*>(w.c.p) + (h / w.c.group) * w.c.head + c0 + (first + t0 + j) * w.c.tok;
                        if (REV ? row <= j : row >= j)
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                if (i + k < cols) o[k] = fmaf(pv, __bfloat162float(cj[i + k]), o[k]);
                    }
                if (i == 48) {
                    tc_fence_before();
                    arrive(&S.o_free[s]);
                }
                const bool wide = KIND != PLAIN && w.out_f32;                     // (forward outputs are bf16)
                if (wide) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        sts128(at_row(lane, (i & 16 ? 4 : 0) + k), __float_as_uint(o[4 * k]), __float_as_uint(o[4 * k + 1]),
                               __float_as_uint(o[4 * k + 2]), __float_as_uint(o[4 * k + 3]));
                } else {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        sts128(at_row(lane, ((i >> 3) & (Q - 1)) + k), bf2(o[8 * k], o[8 * k + 1]), bf2(o[8 * k + 2], o[8 * k + 3]),
                               bf2(o[8 * k + 4], o[8 * k + 5]), bf2(o[8 * k + 6], o[8 * k + 7]));
                }
                if (wide || KIND == PLAIN ? i & 16 : i == 48) {                   // the rows are full
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < Q; ++k) {
                        const int r = RPA * k + rq, col = wide ? i - 16 + 4 * q : (KIND == PLAIN ? i - 16 : 0) + 8 * q;
                        const uint4 v = lds128(at_row(r, q));
                        const int64_t to = ((first + t0 + 32 * I + r) * w.H + h) * w.dc + c0 + col;
                        if (32 * I + r < L && col < cols) {
                            if (wide) *reinterpret_cast<uint4*>(static_cast<float*>(w.out) + to) = v;
                            else *reinterpret_cast<uint4*>(static_cast<bf16*>(w.out) + to) = v;
                        }
                    }
                    __syncwarp();
                }
            }
            if (KIND != PLAIN) {
                fence_async_smem();                       // (the next tile comes by another way)
                arrive(&S.empty_c[s]);
            }
            if (KIND == SPLIT && in) w.dots[((int64_t)blk * w.H + h) * w.rows() + t] = f_inter * (dot.x + dot.y);
        }
    } else if (warp < 16) {
        // ------------------------------------------------------------------------------------------------- state
        const int row = tid & 127, half = (warp - 8) >> 2, k0 = 32 * half;      // row of the state, and of the chunk's tokens
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        float st[32];
        const int64_t state_at = ((int64_t)n * w.H + h) * w.da * w.dc + (int64_t)row * w.s_r + (int64_t)(c0 + k0) * w.s_c;
        // [slot][h][block][columns by four][row][4], of segments and of spans: the rows of a warp side by side
        auto quad = [&](float* state, int i) { return reinterpret_cast<float4*>(state + (int64_t)((k0 + i) / 4 * 128 + row) * 4); };
        float* seg_at = w.seg_states + ((slot * w.H + h) * blocks + blk) * (128 * NB);
        if (w.seg_chunks > 0 && KIND != STATE) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                const float4 v = *quad(seg_at, i);
                st[i] = v.x;
                st[i + 1] = v.y;
                st[i + 2] = v.z;
                st[i + 3] = v.w;
            }
        } else {
            const bool in = KIND != STATE && w.s_in && row < w.da;
            if (w.s_c == 1 && (uintptr_t)w.s_in % 16 == 0) {  // (d_v goes in steps of 8)
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 v = in && k0 + i < cols ? *reinterpret_cast<const float4*>(w.s_in + state_at + i) : make_float4(0.f, 0.f, 0.f, 0.f);
                    st[i] = v.x;
                    st[i + 1] = v.y;
                    st[i + 2] = v.z;
                    st[i + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) st[i] = in && k0 + i < cols ? w.s_in[state_at + (int64_t)i * w.s_c] : 0.f;
            }
        }
        lin::Log2 kept{0.f, 0.f};                         // the log of what is kept of what enters (STATE)
        static_assert(kLinSpan == CK, "a span is a chunk");
        const int64_t slot0 = first / kLinSpan + n;
        auto span_at = [&](int ch) { return w.spans + (((slot0 + ch) * w.H + h) * blocks + blk) * (int64_t)(128 * NB); };
        auto operand = [&] {                              // S as an operand: rows of 64 columns, 128-byte swizzle
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float a = st[8 * i + 2 * k], b = st[8 * i + 2 * k + 1];
                    hi[k] = bf2(a, b);
                    if (KIND == SPLIT) {
                        const F2 l = add2(F2{a, b}, F2{-low(hi[k]), -high(hi[k])});
                        lo[k] = bf2(l.x, l.y);
                    }
                }
                const uint32_t at = row * 128 + (((4 * half + i) ^ (row & 7)) << 4);
                sts128(base + M::S + at, hi[0], hi[1], hi[2], hi[3]);
                if (KIND == SPLIT) sts128(base + M::S + 16384 + at, lo[0], lo[1], lo[2], lo[3]);
            }
            fence_async_smem();
            arrive(&S.s_ready);
        };
        if (KIND != STATE && chunks > 0) operand();
        for (int c = 0; c < chunks; ++c) {
            const int s = c & 1, L = rows_of(c), ch = chunk_of(c);
            const uint32_t tile = base + s * M::STAGE;
            if (KIND == SPLIT && !REV && w.spans) {       // the state goes out (there is always a place; without the question the
                                                          // compiler spills more: backward of B4, T 4096, 16 heads 361 us for 352)
                float* dst = span_at(ch);
#pragma unroll
                for (int i = 0; i < 8; ++i) *quad(dst, 4 * i) = make_float4(st[4 * i], st[4 * i + 1], st[4 * i + 2], st[4 * i + 3]);
            }
            if (!wait(&S.full[s], c >> 1, 32u)) break;
            const float gh = Gh(c)[row], gl = __bfloat162float(Gl(c)[row]), eh = Gh(c)[CK - 1], el = __bfloat162float(Gl(c)[CK - 1]);
            const lin::Keep keep = S.keep[s];
            arrive(&S.gate_empty[s]);
            if (KIND == STATE) kept = lin::add(kept, {eh, el});
            const float f = w.s_state * (REV ? exp2f(gh + gl) : exp2f((eh - gh) + (el - gl)));
            if (KIND == SPLIT && REV) {                   // or is multiplied with the one that did
                float* src = span_at(ch);
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 x = *quad(src, 4 * i);
                    sum = fmaf(st[4 * i], x.x, sum);
                    sum = fmaf(st[4 * i + 1], x.y, sum);
                    sum = fmaf(st[4 * i + 2], x.z, sum);
                    sum = fmaf(st[4 * i + 3], x.w, sum);
                }
                for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
                if (lane == 0)
                    w.anchors[(((slot0 + ch) * w.H + h) * blocks + blk) * 8 + (warp - 8)] = keep.hi * sum;
            }
            if (!wait(&S.full_c[s], c >> 1, 16u)) break;
            uint32_t top = 0;                             // the largest magnitudes
            const bool in = row < L;
            uint4 cv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) cv[i] = lds128(tile + M::C + row * 128 + (((4 * half + i) ^ (row & 7)) << 4));
            if (L < CK && !in)
#pragma unroll
                for (int i = 0; i < 4; ++i) cv[i] = make_uint4(0, 0, 0, 0);
            // f as the sum of two bf16 numbers f1 + f2: c f1 rounds to the first operand, what the rounding left has no more
            // than eight bits and is exact, and c f2 joins it
            const uint32_t f1 = bf2(f, f);
            const float f_rest = f - low(f1);
            const uint32_t f2 = bf2(f_rest, f_rest);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t at = row * 128 + (((4 * half + i) ^ (row & 7)) << 4);
                const uint32_t word[4] = {cv[i].x, cv[i].y, cv[i].z, cv[i].w};
                uint32_t hi[4], lo[4], third[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    top = most(top, word[k]);
                    hi[k] = mul_bf(word[k], f1);
                    const uint32_t rest = fma_bf(word[k], f1, hi[k] ^ 0x80008000u);
                    if (KIND == SPLIT || FINE) {          // (f2 has eight bits too; the decays' gradient wants more)
                        const F2 l = fma2(F2{low(word[k]), high(word[k])}, F2{f_rest, f_rest}, F2{low(rest), high(rest)});
                        lo[k] = bf2(l.x, l.y);
                        if (FINE) {
                            const F2 left = add2(l, F2{-low(lo[k]), -high(lo[k])});
                            third[k] = bf2(left.x, left.y);
                        }
                    } else {
                        lo[k] = fma_bf(word[k], f2, rest);
                    }
                }
                if (FINE) cv[i] = make_uint4(third[0], third[1], third[2], third[3]);
                sts128(base + M::V + at, hi[0], hi[1], hi[2], hi[3]);
                sts128(base + M::V + 16384 + at, lo[0], lo[1], lo[2], lo[3]);
            }
            const bool odd = (top & 0x7F80u) == 0x7F80u || (top & 0x7F800000u) == 0x7F800000u;
            if (odd || !in) {                             // rare: a row to be passed over, or tokens of the next sequence (their
                                                          // scores, which may be under way, are left out in any case)
#pragma unroll
                for (int i = 0; i < 4; ++i) sts128(tile + M::C + row * 128 + (((4 * half + i) ^ (row & 7)) << 4), 0, 0, 0, 0);
                if (!in)
#pragma unroll
                    for (int i = 0; i < 8; ++i) sts128(tile + M::B + half * 16384 + row * 128 + i * 16, 0, 0, 0, 0);
                if (odd)                                  // (the rest of an infinity is no number)
#pragma unroll 1
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t at = base + M::V + 16384 + row * 128 + (((4 * half + i) ^ (row & 7)) << 4);
                        const uint4 lo = lds128(at);
                        const uint32_t word[4] = {lo.x, lo.y, lo.z, lo.w};
                        uint32_t z[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) z[k] = bf2(finite_or_0(low(word[k])), finite_or_0(high(word[k])));
                        sts128(at, z[0], z[1], z[2], z[3]);
                    }
                if (FINE && odd)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t word[4] = {cv[i].x, cv[i].y, cv[i].z, cv[i].w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) word[k] = bf2(finite_or_0(low(word[k])), finite_or_0(high(word[k])));
                        cv[i] = make_uint4(word[0], word[1], word[2], word[3]);
                    }
            }
            const unsigned bits = __ballot_sync(0xffffffffu, odd && in);
            if (lane == 0) S.flags[c & 3][half][warp & 3] = bits;
            fence_async_smem();
            arrive(&S.vhat);
            if (FINE) {                                   // the third part in the state's place, which A S has read
                if (KIND != STATE && !wait(&S.s_read, c, 1u << 13)) break;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sts128(base + M::S + row * 128 + (((4 * half + i) ^ (row & 7)) << 4), cv[i].x, cv[i].y, cv[i].z, cv[i].w);
                fence_async_smem();
                arrive(&S.third);
            }
            if (!wait(&S.ds_full, c, 64u)) break;
            tc_fence_after();
            {
                uint32_t a[2][16], b[2][16];
                tmem_ld16(lanes + M::DS + k0, a[0]);
                tmem_ld16(lanes + M::DS + k0 + 16, a[1]);
                tmem_ld16(lanes + M::DS + 64 + k0, b[0]);
                tmem_ld16(lanes + M::DS + 64 + k0 + 16, b[1]);
                tmem_ld_wait();
                tc_fence_before();
                arrive(&S.ds_free);
#pragma unroll
                for (int k = 0; k < 32; k += 2) {
                    const F2 v = add2(F2{__uint_as_float(a[k >> 4][k & 15]), __uint_as_float(a[k >> 4][(k & 15) + 1])},
                                      F2{__uint_as_float(b[k >> 4][k & 15]), __uint_as_float(b[k >> 4][(k & 15) + 1])});
                    a[k >> 4][k & 15] = __float_as_uint(v.x);
                    a[k >> 4][(k & 15) + 1] = __float_as_uint(v.y);
                }
#pragma unroll
                for (int k = 0; k < 32; k += 2) {
                    const F2 old{st[k], st[k + 1]};
                    const F2 v = fma2(F2{keep.lo, keep.lo}, old, F2{__uint_as_float(a[k >> 4][k & 15]), __uint_as_float(a[k >> 4][(k & 15) + 1])});
                    const F2 now = fma2(F2{keep.hi, keep.hi}, old, v);
                    st[k] = now.x;
                    st[k + 1] = now.y;
                }
            }
            if (KIND != STATE && c + 1 < chunks) operand();
        }
        if (KIND == STATE) {
            mix::wait_behind();                           // (the walk before it enters its segments from the same states)
#pragma unroll
            for (int i = 0; i < 32; i += 4) *quad(seg_at, i) = make_float4(st[i], st[i + 1], st[i + 2], st[i + 3]);
            if (tid == 256 && blk == 0) w.seg_kept[slot * w.H + h] = kept.hi;
        } else if (ok && w.s_out && last && row < w.da) {
            if (w.s_c == 1 && (uintptr_t)w.s_out % 16 == 0) {
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    if (k0 + i < cols) *reinterpret_cast<float4*>(w.s_out + state_at + i) = make_float4(st[i], st[i + 1], st[i + 2], st[i + 3]);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (k0 + i < cols) w.s_out[state_at + (int64_t)i * w.s_c] = st[i];
            }
        }
    } else if (warp == 16) {
        // ------------------------------------------------------------------------------------------- tensor copies
        if (lane == 0 && chunks > 0) {
            prefetch_tmap(&maps.a);
            prefetch_tmap(&maps.b);
            prefetch_tmap(&maps.c);
            const int ha = h / w.a.group, hb = h / w.b.group, hc = h / w.c.group;
            int issued = 0, issued_c = w.test_stall ? chunks : 0;
            uint64_t last = globaltimer_ns();
            // each stream is refilled as soon as what reads its buffer is done: polled, so that none waits behind another
            while (issued < chunks || issued_c < chunks) {
                bool progress = false;
                if (issued < chunks && (issued < 2 || mbar_test(&S.empty[issued & 1], ((issued >> 1) + 1) & 1))) {
                    const int s = issued & 1, t = (int)(first + (int64_t)chunk_of(issued) * CK);
                    uint8_t* tile = smem + s * M::STAGE;
                    mbar_arrive_expect_tx(&S.full[s], KIND == STATE ? 32768 : 65536);
                    for (int i = 0; i < 2; ++i) {
                        if (KIND != STATE) tma_load_3d(tile + M::A + 16384 * i, &maps.a, &S.full[s], 64 * i, ha, t);
                        tma_load_3d(tile + M::B + 16384 * i, &maps.b, &S.full[s], 64 * i, hb, t);
                    }
                    ++issued;
                    progress = true;
                }
                if (issued_c < chunks && (issued_c < 2 || mbar_test(&S.empty_c[issued_c & 1], ((issued_c >> 1) + 1) & 1))) {
                    const int s = issued_c & 1;
                    mbar_arrive_expect_tx(&S.full_c[s], 16384);
                    tma_load_3d(smem + s * M::STAGE + M::C, &maps.c, &S.full_c[s], c0, hc, (int)(first + (int64_t)chunk_of(issued_c) * CK));
                    ++issued_c;
                    progress = true;
                }
                if (progress) {
                    last = globaltimer_ns();
                } else if (globaltimer_ns() - last > kWait) {
                    report(256u);
                    break;
                }
            }
            // what was asked for has landed before the block leaves
            for (int c = issued > 2 ? issued - 2 : 0; c < issued; ++c) mbar_wait(&S.full[c & 1], (c >> 1) & 1, kWait);
            for (int c = issued_c > 2 ? issued_c - 2 : 0; c < issued_c && !w.test_stall; ++c) mbar_wait(&S.full_c[c & 1], (c >> 1) & 1, kWait);
        }
    } else if (warp == 17) {
        // ------------------------------------------------------------------------------------------------ products
        if (chunks > 0) {
            constexpr uint32_t id_raw = idesc_f16(128, 128, true, false, false);   // A (K-major) x B (K-major)
            constexpr uint32_t id_ds = idesc_f16(128, 128, true, true, true);      // B^T (MN-major) x scaled C (MN-major)
            constexpr uint32_t id_third = idesc_f16(128, 64, true, true, true);
            constexpr uint32_t id_oi = idesc_f16(128, 64, true, false, true);      // A (K-major) x S (MN-major); P (TMEM) x C
            const bool wide = w.da > 64;                  // (the second half of the channels is all zeros else)
            const uint64_t v = sdesc(base + M::V, 16384, 1024), so = sdesc(base + M::S, 16384, 1024);
            const uint64_t a0 = sdesc(base + M::A, 16, 1024), b0 = sdesc(base + M::B, 16, 1024);
            const uint64_t bt0 = sdesc(base + M::B, 16384, 1024), c0d = sdesc(base + M::C, 16384, 1024);
            constexpr uint64_t NEXT = M::STAGE / 16;      // (descriptors count in 16 bytes)
            auto scores = [&](int c) {                    // raw = A B^T
                const uint64_t a = a0 + (c & 1) * NEXT, b = b0 + (c & 1) * NEXT;
                const uint32_t d = tmem + M::RAW + (c & 1) * M::RING;
                if (elected()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_f16(d, a + k * 2, b + k * 2, id_raw, k > 0);
                    if (wide)
#pragma unroll
                        for (int k = 0; k < 4; ++k) mma_f16(d, a + 1024 + k * 2, b + 1024 + k * 2, id_raw, 1u);
                    mma_commit(&S.raw_full[c & 1]);
                }
                __syncwarp();
            };
            auto inter = [&](int c) {                     // A S
                if (!wait(&S.s_ready, c, 1u << 14) || (c > 1 && !wait(&S.o_free[c & 1], (c >> 1) - 1, 1u << 15))) return;
                tc_fence_after();
                const uint64_t a = a0 + (c & 1) * NEXT;
                const uint32_t d = tmem + M::OI + (c & 1) * M::OI_RING;
                if (elected()) {
#pragma unroll
                    for (int part = KIND == SPLIT ? 1 : 0; part >= 0; --part) {
                        const uint32_t on = KIND == SPLIT && part == 0;
#pragma unroll
                        for (int k = 0; k < 4; ++k) mma_f16(d, a + k * 2, so + part * 1024 + k * 128, id_oi, on || k > 0);
                        if (wide)
#pragma unroll
                            for (int k = 4; k < 8; ++k) mma_f16(d, a + 1024 + (k - 4) * 2, so + part * 1024 + k * 128, id_oi, 1u);
                    }
                    if (FINE) mma_commit(&S.s_read);
                }
                __syncwarp();
            };
            if (KIND != STATE && wait(&S.full[0], 0, 512u)) {
                tc_fence_after();
                scores(0);
            }
            for (int c = 0; c < chunks && ok; ++c) {
                const int s = c & 1;
                if (KIND != STATE) inter(c);
                if (!ok || !wait(&S.vhat, c, 1u << 11) || (c > 0 && !wait(&S.ds_free, c - 1, 1u << 12))) break;
                tc_fence_after();
                if (FINE) {
                    const uint64_t bt = bt0 + s * NEXT;
                    if (elected())
#pragma unroll
                        for (int k = 0; k < 8; ++k) mma_f16(tmem + M::DS, bt + k * 128, v + k * 128, id_ds, k > 0);
                    __syncwarp();
                    if (!wait(&S.third, c, 1u << 18)) break;
                    tc_fence_after();
                }
                if (elected()) {
                    const uint64_t bt = bt0 + s * NEXT;
#pragma unroll
                    for (int k = 0; k < 8; ++k)           // (the third part onto the second's)
                        if (FINE) mma_f16(tmem + M::DS + 64, bt + k * 128, so + k * 128, id_third, 1u);
                        else mma_f16(tmem + M::DS, bt + k * 128, v + k * 128, id_ds, k > 0);
                    if (KIND == STATE) mma_commit(&S.empty_c[s]);
                    mma_commit(&S.ds_full);               // (of both products: the state's operand has been read too)
                    mma_commit(&S.empty[s]);
                }
                __syncwarp();
                // the next scores and P C, whichever can go first; the scores go into the place of P and P C of the chunk before
                bool next = KIND == STATE || c + 1 == chunks, product = KIND == STATE;
                for (uint64_t t0 = 0; !(next && product);) {
                    bool progress = false;
                    if (!next && __all_sync(0xffffffffu, mbar_test(&S.full[s ^ 1], ((c + 1) >> 1) & 1)) &&
                        (c == 0 || __all_sync(0xffffffffu, mbar_test(&S.o_free[s ^ 1], ((c - 1) >> 1) & 1)))) {
                        tc_fence_after();
                        scores(c + 1);
                        next = progress = true;
                    }
                    if (!product && __all_sync(0xffffffffu, mbar_test(&S.p_ready[s], (c >> 1) & 1))) {
                        tc_fence_after();
                        if (elected()) {                  // P C
                            const uint64_t cm = c0d + s * NEXT;
                            const uint32_t p = tmem + M::P + s * M::RING;
#pragma unroll
                            for (int k = 0; k < 8; ++k) mma_f16_ts(tmem + M::OA + s * M::RING, p + 8 * k, cm + k * 128, id_oi, k > 0);
                            mma_commit(&S.o_full[s]);
                            if (KIND == PLAIN) mma_commit(&S.empty_c[s]);
                        }
                        __syncwarp();
                        product = progress = true;
                    }
                    if (progress) {
                        t0 = 0;
                    } else {
                        const uint64_t now = globaltimer_ns();
                        if (t0 == 0) t0 = now;
                        ok = __all_sync(0xffffffffu, now - t0 <= kWait);
                        if (!ok) {
                            if (lane == 0) report(1u << 16);
                            break;
                        }
                    }
                }
            }
            // every product has completed before the block leaves
            if (ok && KIND == STATE) mbar_wait(&S.ds_full, (chunks - 1) & 1, kWait);
            else if (ok) mbar_wait(&S.o_full[(chunks - 1) & 1], ((chunks - 1) >> 1) & 1, kWait);
        }
    } else if (warp == 18) {
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
            lin::Log2 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const lin::Log2 y = lin::log2_decay(g[i]);
                x[i] = i > 0 ? lin::add(x[i - 1], y) : y;
            }
            fetch(c + 1, g);
            const lin::Log2 all = lin::prefix(x[3], lane);
            lin::Log2 before{__shfl_up_sync(0xffffffffu, all.hi, 1), __shfl_up_sync(0xffffffffu, all.lo, 1)};
            if (lane > 0)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = lin::add(before, x[i]);
            // the first, or last, token of the column block (eight lanes)
            const int at = REV ? lane & 24 : lane | 7;
            const lin::Log2 ref{__shfl_sync(0xffffffffu, x[REV ? 0 : 3].hi, at), __shfl_sync(0xffffffffu, x[REV ? 0 : 3].lo, at)};
            float cf[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) cf[i] = ex2(REV ? lin::minus(x[i], ref) : lin::minus(ref, x[i]));
            const uint32_t lo[2] = {bf2(x[0].lo, x[1].lo), bf2(x[2].lo, x[3].lo)};
            const lin::Keep keep = lin::keep_of({__shfl_sync(0xffffffffu, x[3].hi, 31), __shfl_sync(0xffffffffu, x[3].lo, 31)});
            if (c > 1 && !wait(&S.gate_empty[c & 1], (c >> 1) + 1, 1u << 17)) break;
            reinterpret_cast<float4*>(Gh(c))[lane] = make_float4(x[0].hi, x[1].hi, x[2].hi, x[3].hi);
            reinterpret_cast<float4*>(Cf(c))[lane] = make_float4(cf[0], cf[1], cf[2], cf[3]);
            reinterpret_cast<uint2*>(Gl(c))[lane] = make_uint2(lo[0], lo[1]);
            if (lane == 0) S.keep[c & 1] = keep;
            arrive(&S.full[c & 1]);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    __syncwarp();
    if (warp == 17) tmem_dealloc(tmem, 512);
    last_behind();
}

}  // namespace

bool lin_tensor_fits(const LinWalk& w) {
    auto fits = [](const LinTok& t) { return (uintptr_t)t.p % 16 == 0 && t.tok % 8 == 0 && t.head % 8 == 0; };
    return w.bf16 && w.da <= 128 && w.dc <= 256 && w.dc % 8 == 0 && fits(w.a) && fits(w.b) && fits(w.c) && (!w.x.p || fits(w.x)) &&
           (uintptr_t)w.out % 16 == 0 && device_is_sm100_family();
}

// Chunks of a segment, or 0: all sequences whole.  A chunk takes a walk 2 us and a first pass 1.1, a block 5 us besides, what joins the
// segments and the two launches 12; 152 blocks run at once.  Whole, a walk takes as long as its longest sequence (forward, one of
// 4096 tokens, 4 heads of 128: 64 us, 30 in segments of 4 chunks; of 65,536 tokens, 16 heads: 934 and 398 in segments of 57; two of
// 2048 tokens, 16 heads: 37 and 50).
//
// Of packed sequences the lengths are not known here; the longest is taken to have half of the tokens, and segments are short
// enough to be spread in two or three rounds over the card whatever the lengths (5 sequences, 32,768 tokens, 16 heads, forward and
// backward, one kernel after another: of even lengths 205 and 1025 us whole, 237 and 1006 in segments of 20 chunks; 391 to 13,636
// tokens 207 and 1092, 245 and 1031; one of 30,000 and four short ones 435 and 2138, 237 and 1025).
//
// The generic walk goes by the same rule with its own times: 11 us a chunk and 0.2 us a channel of a, two thirds of that for a first
// pass, blocks that share an SM each at 0.82 of that (forward, fp32: one sequence of 1000 tokens, 16 heads of 128: 291 us whole, 184 in
// segments of one chunk, 178 of two, 290 of four; two of 2048 tokens: 578 whole, 583 of two; two of 777 tokens, 3 heads of 40: 134
// and 50 of one).
int lin_segment_chunks(int64_t rows, int64_t N, bool packed, int H, int da, int dc, bool tensor) {
    if (N < 1 || rows < 1) return 0;
    const int64_t walks = (int64_t)H * lin_blocks(dc, tensor);
    constexpr double BLOCK = 5, JOIN = 12, SMS = 152;
    const double WALK = tensor ? 2 : 11 + 0.195 * da, STATE = tensor ? 1.1 : 0.65 * WALK;
    const int least = tensor ? 4 : 1;                     // chunks of a segment
    // blocks of `each` chunks: in rounds of one an SM, or the generic ones side by side
    auto time = [&](int64_t blocks, int64_t each, double chunk) {
        if (tensor) return (double)((blocks + 151) / 152) * (chunk * each + BLOCK);
        const double full = blocks / SMS, slow = 0.45 + 0.82 * full;
        return chunk * each * (slow > 1 ? slow : 1) + BLOCK * (full > 1 ? full : 1);
    };
    if (packed && N > 1) {
        const double chunks = (double)((rows + CK - 1) / CK), each_sm = chunks * walks / SMS;
        const double each = each_sm / 2.5 < 2 * least ? 2 * least : ceil(each_sm / 2.5);
        const double whole = WALK * (each_sm > chunks / 2 ? each_sm : chunks / 2) + BLOCK;
        return (WALK + STATE) * (each_sm + each / 2) + 2 * BLOCK + JOIN < whole && 2 * each <= chunks ? (int)each : 0;
    }
    const int64_t chunks = (rows / N + CK - 1) / CK;
    double best = time(N * walks, chunks, WALK);
    int best_each = 0;
    for (int64_t n = 2; n <= 64 && least * n <= chunks; ++n) {
        const int64_t each = (chunks + n - 1) / n;
        const double cost = time(N * walks * n, each, WALK) + time(N * walks * (n - 1), each, STATE) + JOIN;
        if (cost < best) {
            best = cost;
            best_each = (int)each;
        }
    }
    return best_each;
}

cudaError_t launch_lin_walk_tensor(const LinWalk& given, bool behind, cudaStream_t s) {
    LinWalk w = given;
    const int blocks = lin_blocks(w.dc, true);
    const int64_t slots = w.seg_chunks > 0 ? lin_slots(w.rows(), w.N(), w.seg_chunks * CK) : w.N();
    const int64_t units = slots * w.H * blocks;
    if (units == 0) return cudaSuccess;
    LinMaps maps{};
    if (w.rows() > 0 && (!token_map(&maps.a, w.a, w.da, w.H / w.a.group, w.rows()) || !token_map(&maps.b, w.b, w.da, w.H / w.b.group, w.rows()) ||
                         !token_map(&maps.c, w.c, w.dc, w.H / w.c.group, w.rows())))
        return cudaErrorInvalidValue;
    auto start = [&](auto kernel, uint32_t smem, bool early) -> cudaError_t {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        return mix::launch_behind(kernel, dim3((unsigned)units), THREADS, smem, early, s, maps, w);
    };
    if (w.seg_chunks > 0) {
        w.wait_first = 0;
        cudaError_t e = w.fine ? w.rev ? start(lin_chunk_kernel<true, STATE, true>, Map<STATE>::BYTES, behind)
                                       : start(lin_chunk_kernel<false, STATE, true>, Map<STATE>::BYTES, behind)
                               : w.rev ? start(lin_chunk_kernel<true, STATE, false>, Map<STATE>::BYTES, behind)
                                       : start(lin_chunk_kernel<false, STATE, false>, Map<STATE>::BYTES, behind);
        if (e == cudaSuccess) e = launch_lin_segments(w, s);
        if (e != cudaSuccess) return e;
        behind = true;
    }
    w.wait_first = behind && (w.spans || w.seg_chunks > 0);
    if (w.dots && w.fine)
        return w.rev ? start(lin_chunk_kernel<true, SPLIT, true>, Map<SPLIT>::BYTES, behind) : start(lin_chunk_kernel<false, SPLIT, true>, Map<SPLIT>::BYTES, behind);
    if (w.dots)
        return w.rev ? start(lin_chunk_kernel<true, SPLIT, false>, Map<SPLIT>::BYTES, behind) : start(lin_chunk_kernel<false, SPLIT, false>, Map<SPLIT>::BYTES, behind);
    return w.rev ? start(lin_chunk_kernel<true, PLAIN, false>, Map<PLAIN>::BYTES, behind) : start(lin_chunk_kernel<false, PLAIN, false>, Map<PLAIN>::BYTES, behind);
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
