// Attention of one new token for each sequence over a paged key-value cache:
//     o = sum_j p_j v_j,   p = softmax_j(scale q . k_j),   j over the sequence's tokens,
// with the running maximum and sum of the softmax in fp32, query heads in groups that share a key and value head.
//
// Bound by reading every key and value once.  The tokens of a sequence are divided into parts (paged_attn_splits), a block of
// four warps for each (sequence, key head, part), and a second kernel joins the parts of a sequence that has more than one.
//
// bf16, head sizes in steps of 8 (as 64, 128 or 256 channels, zeros behind the last), pages, slots and heads of the cache on 16 bytes, q
// on 4, and places within 2^32 pieces of 16 bytes: a warp takes every fourth run of 16 tokens, with no barrier between warps: its own ring of
// STAGES runs in shared memory, filled by 16-byte asynchronous copies (a lane looks up a token's page one run ahead), the
// scores from m16n8k16 products with up to 16 heads of a group as rows, and p as the sum of two bf16 numbers for the product
// with the values (one would add an error as large as the result's own rounding; the second product is hidden behind memory).
// A group has at most 16 rows, an eighth of what the block-wide tensor instructions take, and the products are a tenth of what
// even these warp-wide ones can do beside the bytes, so it is the loads that shape the kernel.
// (256 sequences of up to 8192 tokens, 32 heads over 8 of 128: 650 us, 97 % of the copy rate for the tokens there are; two stages
// and three blocks an SM, or three and two, are the same there.)
// Anything else: a warp a token at a time, lanes along the channels, fp32.

#include <type_traits>

#include "mixer_common.cuh"
#include "paged.h"

namespace gdn {
namespace {

using mix::bf16;
constexpr int WARPS = 4, THREADS = 32 * WARPS, RUN = 16;
constexpr float LOG2E = 1.4426950408889634f;
constexpr int kMaxParts = 1024;

__device__ __forceinline__ int sequence_tokens(const PagedCache& c, int n) {
    const int64_t most = (int64_t)c.max_pages * c.page_size;
    return (int)min(max((int64_t)c.lengths[n], (int64_t)0), min(most, (int64_t)0x7FFFFF00));
}

__device__ __forceinline__ uint32_t smem_at(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
    const int size = in ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {                    // 2^x to 2^-22; 0 below 2^-126
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// two floats as bf16 pairs: the values rounded, and what the rounding left
__device__ __forceinline__ void halves(float x, float y, uint32_t& hi, uint32_t& lo) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    const __nv_bfloat162 l = __floats2bfloat162_rn(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xFFFF0000u));
    lo = *reinterpret_cast<const uint32_t*>(&l);
}

// two bf16 numbers, those that are infinite or no number as 0
__device__ __forceinline__ uint32_t finite_or_0(uint32_t w) {
    return (w & 0x7F80u) == 0x7F80u ? (w & 0x7F800000u) == 0x7F800000u ? 0u : w & 0xFFFF0000u
                                    : (w & 0x7F800000u) == 0x7F800000u ? w & 0xFFFFu : w;
}

// What a block hands on: o (or a part's unscaled sum) of head `hq`, its maximum (base 2) and sum.
struct Part {
    const PagedAttnArgs& a;
    int n, hq, split, parts;
    __device__ float* sums() const { return static_cast<float*>(a.ws) + paged_attn_sums_at(a, n, hq, split); }
    __device__ float* tops() const { return static_cast<float*>(a.ws) + paged_attn_tops_at(a, n, hq, split); }
    template <typename T> __device__ void put(int i, float x, float total) const {
        if (parts > 1) sums()[i] = x;
        else mix::st(static_cast<T*>(a.o) + ((int64_t)n * a.Hq + hq) * a.c.d + i, total > 0.f || total != total ? x / total : 0.f);
    }
    __device__ void close(float top, float total) const {
        if (parts > 1) {
            tops()[0] = top;
            tops()[1] = total;
        } else if (a.lse) {
            a.lse[(int64_t)n * a.Hq + hq] = total > 0.f || total != total ? top / LOG2E + logf(total) : -INFINITY;
        }
    }
};

template <int D, int STAGES>
struct Ring {
    static constexpr int ROW = D * 2 + 16;                 // bytes of a token's row: 16 more, so that eight rows start in different banks
    static constexpr int STAGE = 2 * RUN * ROW, WARP = STAGES * STAGE;
    static constexpr size_t BYTES = (size_t)WARPS * WARP;
};

template <int D, int STAGES>
__global__ void __launch_bounds__(THREADS, D == 64 ? 4 : D == 128 ? 3 : 1) paged_attn_mma_kernel(const PagedAttnArgs a) {
    using R = Ring<D, STAGES>;
    extern __shared__ __align__(16) char ring[];
    __shared__ float top_s[WARPS][16], sum_s[WARPS][16];
    const PagedCache& c = a.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = a.Hq / c.Hk, tiles = (group + 15) / 16;
    int64_t unit = blockIdx.x;                         // (key heads first: their rows lie side by side)
    const int hk = (int)(unit % c.Hk);
    unit /= c.Hk;
    const int tile = (int)(unit % tiles);
    unit /= tiles;
    const int split = (int)(unit % a.splits), n = (int)(unit / a.splits);
    const int len = sequence_tokens(c, n), per = paged_attn_part_tokens(len, a.splits), parts = paged_attn_parts(len, per);
    const int t0 = paged_attn_part_begin(len, per, split), t1 = paged_attn_part_begin(len, per, split + 1);
    mix::let_next();
    if (t0 >= t1 && split > 0) return;
    const int rows = min(16, group - tile * 16), hq0 = hk * group + tile * 16;

    // q as the products' first operand: rows are heads
    uint32_t q[D / 16][4];
    {
        const bf16* src = static_cast<const bf16*>(a.q) + n * a.q_tok + (int64_t)hq0 * a.q_head;
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = lane / 4 + (i & 1) * 8, at = s * 16 + (i >> 1) * 8 + lane % 4 * 2;
                q[s][i] = r < rows && at < c.d ? *reinterpret_cast<const uint32_t*>(src + r * a.q_head + at) : 0u;
            }
    }
    const int runs = (t1 - t0 + RUN - 1) / RUN, mine = runs > warp ? (runs - warp + WARPS - 1) / WARPS : 0;
    const uint32_t base = smem_at(ring) + warp * R::WARP;
    const bf16* kp = static_cast<const bf16*>(c.k.p) + hk * c.k.head;
    const bf16* vp = static_cast<const bf16*>(c.v.p) + hk * c.v.head;
    // lane l (and l + 16): where token l of a run lies, in 16 bytes from the first key (value), and whether it does
    struct Where { uint32_t k, v; bool in; };
    auto look_up = [&](int run) {
        Where at{0, 0, false};
        if (run >= mine) return at;                                // (past the part, and maybe past 31 bits)
        const int t = t0 + (warp + run * WARPS) * RUN + (lane & 15);
        if (t < t1) {
            const int page = c.table[n * c.table_ld + t / c.page_size], slot = t % c.page_size;
            at.in = page >= 0 && page < c.n_pages;
            if (at.in) {
                at.k = (uint32_t)((page * c.k.page + slot * c.k.slot) / 8);
                at.v = (uint32_t)((page * c.v.page + slot * c.v.slot) / 8);
            }
        }
        return at;
    };
    auto fill = [&](int run, const Where& at, unsigned in) {
        if (run < mine) {
            constexpr int PER = D / 8, EACH = RUN * PER / 32;      // 16-byte pieces of a row; those of a lane
            const int col = lane % PER;
            const uint32_t dst = base + (run % STAGES) * R::STAGE + lane / PER * R::ROW + col * 16;
            const bool wide = col * 8 < c.d;
#pragma unroll
            for (int u = 0; u < EACH; ++u) {
                const int r = u * (32 / PER) + lane / PER;
                const uint32_t ko = __shfl_sync(0xffffffffu, at.k, r), vo = __shfl_sync(0xffffffffu, at.v, r);
                const bool have = wide && (in >> r) & 1;
                copy16(dst + u * (32 / PER) * R::ROW, kp + (have ? (uint64_t)ko * 8 + col * 8 : 0), have);
                copy16(dst + (RUN + u * (32 / PER)) * R::ROW, vp + (have ? (uint64_t)vo * 8 + col * 8 : 0), have);
            }
        }
        mix::copies_close();
    };

    // An infinite value is p infinities.  But the second of the two numbers that p is may be 0 or negative, and the sum of both
    // products then no number; so where that is what came out, the warp takes its tokens once more, with values that are not
    // finite left out of the second product.
    float o[D / 8][4], top[2], sum[2];
    auto take = [&](auto apart) {
        top[0] = top[1] = -INFINITY;
        sum[0] = sum[1] = 0.f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
        // which tokens of a run are there: a bit each, in the order of the runs (STAGES runs are on their way)
        unsigned there[STAGES];
        Where at = look_up(0);
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s) {
            const Where ahead = look_up(s + 1);
            there[s] = __ballot_sync(0xffffffffu, at.in) & 0xFFFFu;
            fill(s, at, there[s]);
            at = ahead;
        }
        const float scale = a.scale * LOG2E;
        for (int run0 = 0; run0 < mine; run0 += STAGES)
#pragma unroll
            for (int st = 0; st < STAGES; ++st) {
                const int run = run0 + st;
                if (run >= mine) break;
                mix::copies_wait<STAGES - 2>();
                __syncwarp();                                          // (every lane's copies have landed, and the stage filled next is read)
                constexpr int LAST = STAGES - 1;
                {
                    const Where ahead = look_up(run + STAGES);
                    there[(st + LAST) % STAGES] = __ballot_sync(0xffffffffu, at.in) & 0xFFFFu;
                    fill(run + LAST, at, there[(st + LAST) % STAGES]);
                    at = ahead;
                }
                const uint32_t ks = base + st * R::STAGE, vs = ks + RUN * R::ROW;
                float x[2][4] = {};                                    // heads lane / 4 and + 8, tokens 8 i + lane % 4 * 2 and + 1
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    uint32_t b[4];                                     // tokens 0-7 and 8-15, channels 0-7 and 8-15 of the step
                    ldsm4(b, ks + (lane % 8 + (lane >> 4) * 8) * R::ROW + s * 32 + ((lane >> 3) & 1) * 16);
                    mma16816(x[0], q[s], b[0], b[1]);
                    mma16816(x[1], q[s], b[2], b[3]);
                }
                const unsigned live = there[st];
                float most[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x[i][j] *= scale;
                        if (live != 0xFFFFu && !((live >> (8 * i + lane % 4 * 2 + (j & 1))) & 1)) x[i][j] = -INFINITY;
                        most[j >> 1] = fmaxf(most[j >> 1], x[i][j]);
                    }
                bool more = false;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    most[r] = fmaxf(most[r], __shfl_xor_sync(0xffffffffu, most[r], 1));
                    most[r] = fmaxf(most[r], __shfl_xor_sync(0xffffffffu, most[r], 2));
                    more |= most[r] > top[r];
                }
                if (__any_sync(0xffffffffu, more)) {
                    float f[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float now = fmaxf(top[r], most[r]);
                        f[r] = top[r] == now ? 1.f : exp2f(top[r] - now);
                        top[r] = now;
                        sum[r] *= f[r];
                    }
#pragma unroll
                    for (int i = 0; i < D / 8; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) o[i][j] *= f[j >> 1];
                }
                const float zero[2] = {top[0] == -INFINITY ? 0.f : top[0], top[1] == -INFINITY ? 0.f : top[1]};
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x[i][j] = ex2(x[i][j] - zero[j >> 1]);
                        sum[j >> 1] += x[i][j];
                    }
                uint32_t hi[4], lo[4];
                halves(x[0][0], x[0][1], hi[0], lo[0]);
                halves(x[0][2], x[0][3], hi[1], lo[1]);
                halves(x[1][0], x[1][1], hi[2], lo[2]);
                halves(x[1][2], x[1][3], hi[3], lo[3]);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    uint32_t b[4];                                     // tokens 0-7, 8-15 of channels 0-7, then of channels 8-15
                    ldsm4_t(b, vs + (lane % 16) * R::ROW + i * 32 + (lane >> 4) * 16);
                    mma16816(o[2 * i], hi, b[0], b[1]);
                    mma16816(o[2 * i + 1], hi, b[2], b[3]);
                    if (apart.value)
#pragma unroll
                        for (int k = 0; k < 4; ++k) b[k] = finite_or_0(b[k]);
                    mma16816(o[2 * i], lo, b[0], b[1]);
                    mma16816(o[2 * i + 1], lo, b[2], b[3]);
                }
            }
        mix::copies_wait<0>();
        __syncwarp();
    };
    take(std::false_type{});
    bool nan = false;
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) nan |= o[i][j] != o[i][j];
    if (__any_sync(0xffffffffu, nan)) take(std::true_type{});
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
        sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
    }
    if (lane % 4 == 0)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            top_s[warp][lane / 4 + 8 * r] = top[r];
            sum_s[warp][lane / 4 + 8 * r] = sum[r];
        }
    __syncthreads();
    // the warps' parts join in shared memory, each brought to the common maximum
    float* joint = reinterpret_cast<float*>(ring);                 // [WARPS][16][D]
    float f[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = lane / 4 + 8 * r;
        float all = -INFINITY;
        for (int w = 0; w < WARPS; ++w) all = fmaxf(all, top_s[w][row]);
        f[r] = top[r] == all ? 1.f : exp2f(top[r] - all);
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r)
            *reinterpret_cast<float2*>(joint + (warp * 16 + lane / 4 + 8 * r) * D + i * 8 + lane % 4 * 2) =
                make_float2(f[r] * o[i][2 * r], f[r] * o[i][2 * r + 1]);
    __syncthreads();
    for (int row = warp; row < rows; row += WARPS) {
        float all = -INFINITY, total = 0.f;
        for (int w = 0; w < WARPS; ++w) all = fmaxf(all, top_s[w][row]);
        for (int w = 0; w < WARPS; ++w) total += sum_s[w][row] * (top_s[w][row] == all ? 1.f : exp2f(top_s[w][row] - all));
        const Part part{a, n, hq0 + row, split, parts};
        for (int i = lane; i < c.d; i += 32) {
            float s = 0.f;
            for (int w = 0; w < WARPS; ++w) s += joint[(w * 16 + row) * D + i];
            part.put<bf16>(i, s, total);
        }
        if (lane == 0) part.close(all, total);
    }
}

// Any type, head size up to 256 and alignment: HEADS heads of a group at a time, lanes along the channels.
constexpr int HEADS = 4, CHAN = 8;
template <typename T>
__global__ void __launch_bounds__(THREADS) paged_attn_generic_kernel(const PagedAttnArgs a) {
    __shared__ float top_s[WARPS][HEADS], sum_s[WARPS][HEADS], joint[WARPS][HEADS][256];
    const PagedCache& c = a.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = a.Hq / c.Hk, tiles = (group + HEADS - 1) / HEADS;
    int64_t unit = blockIdx.x;                         // (key heads first: their rows lie side by side)
    const int hk = (int)(unit % c.Hk);
    unit /= c.Hk;
    const int tile = (int)(unit % tiles);
    unit /= tiles;
    const int split = (int)(unit % a.splits), n = (int)(unit / a.splits);
    const int len = sequence_tokens(c, n), per = paged_attn_part_tokens(len, a.splits), parts = paged_attn_parts(len, per);
    const int t0 = paged_attn_part_begin(len, per, split), t1 = paged_attn_part_begin(len, per, split + 1);
    mix::let_next();
    if (t0 >= t1 && split > 0) return;
    const int heads = min(HEADS, group - tile * HEADS), hq0 = hk * group + tile * HEADS;
    const T* qp = static_cast<const T*>(a.q) + n * a.q_tok + (int64_t)hq0 * a.q_head;
    const T* kp = static_cast<const T*>(c.k.p) + hk * c.k.head;
    const T* vp = static_cast<const T*>(c.v.p) + hk * c.v.head;
    float q[HEADS][CHAN], o[HEADS][CHAN], top[HEADS], sum[HEADS];
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
        top[h] = -INFINITY;
        sum[h] = 0.f;
#pragma unroll
        for (int i = 0; i < CHAN; ++i) {
            const int at = lane + 32 * i;
            q[h][i] = h < heads && at < c.d ? mix::ld(qp + h * a.q_head + at) : 0.f;
            o[h][i] = 0.f;
        }
    }
    const float scale = a.scale * LOG2E;
    constexpr int AT_ONCE = 2;                                     // tokens of a warp whose reads are in flight together
    for (int t = t0 + warp * AT_ONCE; t < t1; t += WARPS * AT_ONCE) {
        float k[AT_ONCE][CHAN], v[AT_ONCE][CHAN];
        bool in[AT_ONCE];
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) {
            int64_t page = t + u < t1 ? c.table[n * c.table_ld + (t + u) / c.page_size] : -1;
            in[u] = page >= 0 && page < c.n_pages;
            if (!in[u]) page = 0;
            const int64_t slot = (t + u) % c.page_size;
#pragma unroll
            for (int i = 0; i < CHAN; ++i) {
                const int at = lane + 32 * i;
                const bool have = in[u] && at < c.d;
                k[u][i] = have ? mix::ld(kp + page * c.k.page + slot * c.k.slot + at) : 0.f;
                v[u][i] = have ? mix::ld(vp + page * c.v.page + slot * c.v.slot + at) : 0.f;
            }
        }
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) {
            if (!in[u]) continue;
#pragma unroll
            for (int h = 0; h < HEADS; ++h) {
                if (h >= heads) break;
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < CHAN; ++i) s = fmaf(q[h][i], k[u][i], s);
                for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
                s *= scale;
                if (s > top[h]) {
                    const float f = exp2f(top[h] - s);
                    top[h] = s;
                    sum[h] *= f;
#pragma unroll
                    for (int i = 0; i < CHAN; ++i) o[h][i] *= f;
                }
                const float p = exp2f(s - (top[h] == -INFINITY ? 0.f : top[h]));
                sum[h] += p;
#pragma unroll
                for (int i = 0; i < CHAN; ++i) o[h][i] = fmaf(p, v[u][i], o[h][i]);
            }
        }
    }
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
        if (lane == 0) {
            top_s[warp][h] = top[h];
            sum_s[warp][h] = sum[h];
        }
#pragma unroll
        for (int i = 0; i < CHAN; ++i) joint[warp][h][lane + 32 * i] = o[h][i];
    }
    __syncthreads();
    for (int h = warp; h < heads; h += WARPS) {
        float all = -INFINITY, total = 0.f, f[WARPS];
        for (int w = 0; w < WARPS; ++w) all = fmaxf(all, top_s[w][h]);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            f[w] = top_s[w][h] == all ? 1.f : exp2f(top_s[w][h] - all);
            total += sum_s[w][h] * f[w];
        }
        const Part part{a, n, hq0 + h, split, parts};
        for (int i = lane; i < c.d; i += 32) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) s = fmaf(f[w], joint[w][h][i], s);
            part.put<T>(i, s, total);
        }
        if (lane == 0) part.close(all, total);
    }
}

// Joins the parts of each (sequence, query head) that has more than one: a block each, a channel a thread.
template <typename T>
__global__ void __launch_bounds__(THREADS) paged_attn_join_kernel(const PagedAttnArgs a) {
    __shared__ float tops_s[kMaxParts], sums_s[kMaxParts];
    const PagedCache& c = a.c;
    const int tid = threadIdx.x, lane = tid & 31;
    const int n = blockIdx.x / a.Hq, hq = blockIdx.x % a.Hq;
    const int len = sequence_tokens(c, n), parts = paged_attn_parts(len, paged_attn_part_tokens(len, a.splits));
    mix::wait_behind();
    if (parts <= 1) return;
    const float* sums = Part{a, n, hq, 0, parts}.sums();
    const float* tops = Part{a, n, hq, 0, parts}.tops();
    for (int s = tid; s < parts; s += THREADS) {
        const float2 t = *reinterpret_cast<const float2*>(tops + 2 * s);
        tops_s[s] = t.x;
        sums_s[s] = t.y;
    }
    __syncthreads();
    float top = -INFINITY;
    for (int s = lane; s < parts; s += 32) top = fmaxf(top, tops_s[s]);
    for (int m = 16; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
    __syncthreads();
    for (int s = tid; s < parts; s += THREADS) tops_s[s] = tops_s[s] == top ? 1.f : exp2f(tops_s[s] - top);
    __syncthreads();
    float total = 0.f, o[2] = {0.f, 0.f};
    const bool in[2] = {tid < c.d, tid + THREADS < c.d};
    for (int s0 = 0; s0 < parts; s0 += 8) {                        // eight parts' reads on their way
        float x[8][2];
#pragma unroll
        for (int u = 0; u < 8; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i) x[u][i] = s0 + u < parts && in[i] ? sums[(int64_t)(s0 + u) * c.d + tid + i * THREADS] : 0.f;
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (s0 + u < parts) {
                const float f = tops_s[s0 + u];
                total = fmaf(f, sums_s[s0 + u], total);
                o[0] = fmaf(f, x[u][0], o[0]);
                o[1] = fmaf(f, x[u][1], o[1]);
            }
    }
    const Part part{a, n, hq, 0, 1};
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (in[i]) part.put<T>(tid + i * THREADS, o[i], total);
    if (tid == 0) part.close(top, total);
}

template <int D, int STAGES>
cudaError_t start_mma(const PagedAttnArgs& a, unsigned blocks, cudaStream_t s) {
    constexpr size_t joint = (size_t)WARPS * 16 * D * 4;
    constexpr size_t smem = Ring<D, STAGES>::BYTES > joint ? Ring<D, STAGES>::BYTES : joint;
    const cudaError_t e = cudaFuncSetAttribute(paged_attn_mma_kernel<D, STAGES>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    paged_attn_mma_kernel<D, STAGES><<<blocks, THREADS, smem, s>>>(a);
    return cudaGetLastError();
}

bool vector_rows(const PagedAttnArgs& a) {
    auto fits = [](const PagedSide& x) { return (uintptr_t)x.p % 16 == 0 && x.page % 8 == 0 && x.slot % 8 == 0 && x.head % 8 == 0; };
    // (a row's place is counted in 16 bytes and 32 bits)
    auto near = [&](const PagedSide& x) { return (a.c.n_pages * x.page + a.c.page_size * x.slot) / 8 < (int64_t(1) << 32); };
    return a.c.bf16 && near(a.c.k) && near(a.c.v) && a.c.d % 8 == 0 && fits(a.c.k) && fits(a.c.v) && (uintptr_t)a.q % 4 == 0 && a.q_tok % 2 == 0 && a.q_head % 2 == 0;
}

}  // namespace

// As many parts as give two blocks an SM (of 152) with full sequences (one sequence of 32,768 tokens, 32 heads over 8: 34.9 us; for the
// three that fit an SM 36.9, the join takes longer), none smaller than 128 tokens or (where there are blocks
// enough without, so that long sequences of a ragged batch do not run last and alone) larger than 2048.  Lengths are on the device, so
// all this goes by the table's width, and a sequence far shorter than that is in parts of 128 tokens: 256 sequences of up to 8192 tokens
// take 628 us with a table of 8192, 753 of 32,768 and 1169 of 131,072; 32 of 2048 tokens 66 us, and 88 of 32,768.
int paged_attn_splits(const PagedAttnArgs& a) {
    const int64_t most = (int64_t)a.c.max_pages * a.c.page_size;
    const int group = a.Hq / a.c.Hk, tiles = (group + 15) / 16;
    const int64_t units = (int64_t)a.c.N * a.c.Hk * tiles;
    const int64_t least = (most + 2047) / 2048, fill = 304 / (units > 0 ? units : 1), top = (most + 127) / 128;
    int64_t s = least > fill ? least : fill;
    if (s > top) s = top;
    return (int)(s < 1 ? 1 : s > kMaxParts ? kMaxParts : s);
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t s) {
    const int group = a.Hq / a.c.Hk;
    cudaError_t e;
    if (vector_rows(a)) {
        const unsigned blocks = (unsigned)((int64_t)a.c.N * a.c.Hk * ((group + 15) / 16) * a.splits);
        if (a.c.d <= 64) e = start_mma<64, 3>(a, blocks, s);
        else if (a.c.d <= 128) e = start_mma<128, 2>(a, blocks, s);
        else e = start_mma<256, 3>(a, blocks, s);
    } else {
        const unsigned blocks = (unsigned)((int64_t)a.c.N * a.c.Hk * ((group + HEADS - 1) / HEADS) * a.splits);
        if (a.c.bf16) paged_attn_generic_kernel<bf16><<<blocks, THREADS, 0, s>>>(a);
        else paged_attn_generic_kernel<float><<<blocks, THREADS, 0, s>>>(a);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess || a.splits <= 1) return e;
    const unsigned blocks = (unsigned)((int64_t)a.c.N * a.Hq);
    return a.c.bf16 ? mix::launch_behind(paged_attn_join_kernel<bf16>, blocks, THREADS, 0, true, s, a)
                    : mix::launch_behind(paged_attn_join_kernel<float>, blocks, THREADS, 0, true, s, a);
}

}  // namespace gdn
