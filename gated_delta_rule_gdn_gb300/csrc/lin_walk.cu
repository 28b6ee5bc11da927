// Linear attention with a decay for each head: the generic walk (fp32 arithmetic, any head size up to 256, fp32 or bf16
// tokens), and the sums behind the walks of the backward pass.
//
// One block of threads walks one (sequence, value head, 32 columns of c) in chunks of 32 tokens, with the state in shared
// memory.  Half of its warps bring the next chunk's rows (and the prefix sums of its decays) while the others work: the 32 x 32
// triangle of decayed products a_i . b_j, the outputs (row i: a_i S and the triangle's row), then the state.  Bound by reads of
// shared memory, so a thread takes four rows at a time, and four channels an access (2 sequences of 777 tokens, 3 heads of 40, fp32,
// forward and backward: 1.30 ms a channel and a row at a time, 0.64 so, 0.18 in segments; what is left is one block's latency).  The
// triangle is a loop bound, not a factor, so a value that is not a number reaches no token it should not.

#include "internal.h"
#include "lin_common.cuh"

namespace gdn {
namespace {

using mix::bf16;
constexpr int CH = kLinGenericChunk, COLS = kLinGenericCols, WORK = 256, THREADS = 2 * WORK, WARPS = WORK / 32;

// A chunk's rows in fp32, tokens behind the sequence as zeros, and its decays.
struct GenericTile {
    float *A, *B, *C, *X;                              // [CH][lda] twice (zeros up to a step of four channels), [CH][COLS] twice
    lin::Log2* G;
    float *rowf, *colf;
    lin::Keep* keep;
};
__host__ __device__ inline int four(int n) { return (n + 3) & ~3; }
// 4 more than a multiple of 32: 16-byte reads of eight rows at one column hit different banks
__host__ __device__ inline int generic_lda(int da) { return (four(da) + 27) / 32 * 32 + 4; }
__host__ __device__ inline size_t generic_tile_floats(int da) { return 2 * (size_t)CH * generic_lda(da) + 2 * CH * COLS + 4 * CH + 4; }
constexpr int PLD = CH + 4;                            // row of the triangle

// STATE: the state alone, of a segment from nothing.
template <typename T, bool STATE>
__global__ void __launch_bounds__(THREADS, 2) lin_walk_kernel(const LinWalk w) {
    mix::let_next();
    if (w.wait_first) mix::wait_behind();
    extern __shared__ __align__(16) float sh[];
    const int da = w.da, da4 = four(da), lda = generic_lda(da);
    float* S = sh;                                     // [da4][COLS]
    float* P = S + da4 * COLS;                         // [CH][PLD], decays and all
    float* tiles = P + CH * PLD;
    auto tile = [&](int k) {
        GenericTile t;
        float* p = tiles + (k & 1) * generic_tile_floats(da);
        t.G = reinterpret_cast<lin::Log2*>(p);
        t.rowf = p + 2 * CH;
        t.colf = t.rowf + CH;
        t.keep = reinterpret_cast<lin::Keep*>(t.colf + CH);          // (two words)
        t.A = t.colf + CH + 4;
        t.B = t.A + CH * lda;
        t.C = t.B + CH * lda;
        t.X = t.C + CH * COLS;
        return t;
    };
    __shared__ float red[WARPS];
    constexpr int R = CH / WARPS;                      // rows of a warp

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int blocks = (w.dc + COLS - 1) / COLS;
    const int64_t unit = blockIdx.x;
    const int blk = (int)(unit % blocks), h = (int)(unit / blocks % w.H);
    const int64_t slot = unit / blocks / w.H;          // a sequence, or a segment of one
    int64_t first;
    int n, len, base = 0, chunks;                      // base: the segment's first token
    bool last = true;                                  // in the walk's direction
    if (w.seg_chunks > 0) {
        const int size = w.seg_chunks * kLinChunk;
        n = lin::slot_sequence(w.cu, w.N(), w.T, size, slot);
        lin::sequence(w.cu, w.T, n, first, len);
        const int64_t at = (slot - (first / size + n)) * size;
        if (at >= 0 && at < len) {
            base = (int)at;
            last = w.rev ? at == 0 : at + size >= len;
        }
        if (at < 0 || at >= len || (STATE && last)) {  // (no segment; or none enters behind it)
            lin::last_behind();
            return;
        }
        chunks = (min(size, len - base) + CH - 1) / CH;
    } else {
        n = lin::by_length(w.cu, w.n_seqs, w.T, (int)slot);
        lin::sequence(w.cu, w.T, n, first, len);
        chunks = (len + CH - 1) / CH;
    }
    const int c0 = blk * COLS, cols = min(COLS, w.dc - c0);
    const T* a = static_cast<const T*>(w.a.p) + (h / w.a.group) * w.a.head;
    const T* b = static_cast<const T*>(w.b.p) + (h / w.b.group) * w.b.head;
    const T* c = static_cast<const T*>(w.c.p) + (h / w.c.group) * w.c.head + c0;
    const T* x = w.dots ? static_cast<const T*>(w.x.p) + (h / w.x.group) * w.x.head + c0 : nullptr;
    const int64_t slot0 = first / kLinSpan + n;
    const int64_t state0 = ((int64_t)n * w.H + h) * da * w.dc;
    auto at_state = [&](int r, int cc) { return state0 + (int64_t)r * w.s_r + (int64_t)(c0 + cc) * w.s_c; };

    float* seg_at = w.seg_states + ((slot * w.H + h) * blocks + blk) * ((int64_t)da * COLS);
    for (int e = da * COLS + tid; e < da4 * COLS; e += THREADS) S[e] = 0.f;
    for (int e = tid; e < da * COLS; e += THREADS) {
        if (STATE || w.seg_chunks > 0) {
            S[e] = STATE ? 0.f : seg_at[e];
            continue;
        }
        // (neighbouring threads along the dimension that is contiguous in memory)
        const int r = w.s_c == 1 ? e / COLS : e % da, cc = w.s_c == 1 ? e % COLS : e / da;
        S[r * COLS + cc] = w.s_in && cc < cols ? w.s_in[at_state(r, cc)] : 0.f;
    }

    lin::Log2 all{0.f, 0.f};                           // the log of what is kept of what enters (STATE)
    auto start_of = [&](int step) { return base + (w.rev ? chunks - 1 - step : step) * CH; };
    // a chunk's rows by one half of the warps, a warp a row
    auto bring = [&](int step) {
        const GenericTile t = tile(step);
        const int t0 = start_of(step), L = min(CH, len - t0), wp = warp & (WARPS - 1);
        if (wp == WARPS - 1) {                         // prefix sums of the log decays
            const lin::Log2 s = lin::prefix(lane < L ? lin::log2_decay(w.g[(first + t0 + lane) * w.g_tok + h * w.g_head]) : lin::Log2{0.f, 0.f}, lane);
            const lin::Log2 end{__shfl_sync(0xffffffffu, s.hi, 31), __shfl_sync(0xffffffffu, s.lo, 31)};
            const float before = exp2f(s.hi + s.lo), behind = exp2f(lin::minus(end, s));
            t.G[lane] = s;
            t.rowf[lane] = w.s_inter * (w.rev ? behind : before);
            t.colf[lane] = w.s_state * (w.rev ? before : behind);
            if (lane == 0) *t.keep = lin::keep_of(end);
        }
        const int64_t row = first + t0;                // (all of a lane's rows are on their way before the first is put down)
        float y[R], z[R];
        for (int r = lane; r < da4; r += 32) {
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const int i = r < da ? wp + k * WARPS : CH;
                y[k] = !STATE && i < L ? mix::ld(a + (row + i) * w.a.tok + r) : 0.f;
                z[k] = i < L ? mix::ld(b + (row + i) * w.b.tok + r) : 0.f;
            }
#pragma unroll
            for (int k = 0; k < R; ++k) {
                if (!STATE) t.A[(wp + k * WARPS) * lda + r] = y[k];
                t.B[(wp + k * WARPS) * lda + r] = z[k];
            }
        }
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int i = wp + k * WARPS;
            const bool in = i < L && lane < cols;
            y[k] = in ? mix::ld(c + (row + i) * w.c.tok + lane) : 0.f;
            z[k] = !STATE && in && x ? mix::ld(x + (row + i) * w.x.tok + lane) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < R; ++k) {
            t.C[(wp + k * WARPS) * COLS + lane] = y[k];
            if (!STATE) t.X[(wp + k * WARPS) * COLS + lane] = z[k];
        }
    };
    if (warp >= WARPS && chunks > 0) bring(0);
    __syncthreads();

    auto work_sync = [] { asm volatile("bar.sync 1, 256;" ::: "memory"); };
    for (int step = 0; step < chunks; ++step) {
        if (warp >= WARPS) {
            if (step + 1 < chunks) bring(step + 1);
        } else {
            const GenericTile t = tile(step);
            const int t0 = start_of(step), L = min(CH, len - t0);
            // a span's first chunk: the state goes out, or is multiplied with the one that did
            const bool starts_span = !STATE && w.spans && t0 % kLinSpan == 0;
            const int64_t span = ((slot0 + t0 / kLinSpan) * w.H + h) * blocks + blk;
            if (starts_span && !w.rev)
                for (int e = tid; e < da * COLS; e += WORK) w.spans[span * (da * COLS) + e] = S[e];
            float s[R] = {}, f[R] = {};
            auto at4 = [](const float* p) { return *reinterpret_cast<const float4*>(p); };
            if (!STATE) {
#pragma unroll 2
                for (int r = 0; r < da4; r += 4) {         // row i = warp + k WARPS, column j = lane
                    const float4 y = at4(t.B + lane * lda + r);
#pragma unroll
                    for (int k = 0; k < R; ++k) {
                        const float4 u = at4(t.A + (warp + k * WARPS) * lda + r);
                        s[k] = fmaf(u.w, y.w, fmaf(u.z, y.z, fmaf(u.y, y.y, fmaf(u.x, y.x, s[k]))));
                    }
                }
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    const int i = warp + k * WARPS;
                    const bool pair = w.rev ? lane >= i : lane <= i;
                    if (pair) P[i * PLD + lane] = w.s_intra * s[k] * exp2f(w.rev ? lin::minus(t.G[lane], t.G[i]) : lin::minus(t.G[i], t.G[lane]));
                    s[k] = 0.f;
                }
                __syncwarp();                              // (a warp reads its own rows of P)
#pragma unroll 2
                for (int r = 0; r < da4; r += 4) {         // a warp its rows, a lane a column
                    const float y[4] = {S[r * COLS + lane], S[(r + 1) * COLS + lane], S[(r + 2) * COLS + lane], S[(r + 3) * COLS + lane]};
#pragma unroll
                    for (int k = 0; k < R; ++k) {
                        const float4 u = at4(t.A + (warp + k * WARPS) * lda + r);
                        s[k] = fmaf(u.w, y[3], fmaf(u.z, y[2], fmaf(u.y, y[1], fmaf(u.x, y[0], s[k]))));
                    }
                }
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    const int i = warp + k * WARPS, j1 = w.rev ? L : i;
                    int j = w.rev ? i + 1 : 0;
                    for (; j < j1 && (j & 3); ++j) f[k] = fmaf(P[i * PLD + j], t.C[j * COLS + lane], f[k]);
                    for (; j + 4 <= j1; j += 4) {
                        const float4 u = at4(P + i * PLD + j);
                        const float* y = t.C + j * COLS + lane;
                        f[k] = fmaf(u.w, y[3 * COLS], fmaf(u.z, y[2 * COLS], fmaf(u.y, y[COLS], fmaf(u.x, y[0], f[k]))));
                    }
                    for (; j < j1; ++j) f[k] = fmaf(P[i * PLD + j], t.C[j * COLS + lane], f[k]);
                }
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    const int i = warp + k * WARPS;
                    if (i >= L) continue;
                    const int64_t row = first + t0 + i;
                    float y = s[k] * t.rowf[i];
                    if (w.dots) {
                        const float xi = t.X[i * COLS + lane];
                        float d = lane < cols ? xi * y : 0.f, p = lane < cols ? xi * f[k] : 0.f;
                        for (int m = 16; m > 0; m >>= 1) {
                            d += __shfl_xor_sync(0xffffffffu, d, m);
                            p += __shfl_xor_sync(0xffffffffu, p, m);
                        }
                        if (lane == 0) {
                            w.dots[((int64_t)blk * w.H + h) * w.rows() + row] = d;
                            w.pair_dots[((int64_t)blk * w.H + h) * w.rows() + row] = p;
                        }
                    }
                    y = fmaf(P[i * PLD + i], t.C[i * COLS + lane], y + f[k]);
                    if (lane < cols) {
                        const int64_t at = (row * w.H + h) * w.dc + c0 + lane;
                        if (w.out_f32) static_cast<float*>(w.out)[at] = y;
                        else mix::st(static_cast<T*>(w.out) + at, y);
                    }
                }
            } else if (tid == 0) {
                all = lin::add(all, t.G[CH - 1]);
            }
            const lin::Keep kept = *t.keep;
            if (starts_span && w.rev) {
                float sum = 0.f;
                for (int e = tid; e < da * COLS; e += WORK) sum = fmaf(S[e], w.spans[span * (da * COLS) + e], sum);
                for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
                if (lane == 0) red[warp] = sum;
            }
            work_sync();                               // every row has read the state
            if (starts_span && w.rev && tid == 0) {
                float sum = 0.f;
                for (int i = 0; i < WARPS; ++i) sum += red[i];
                w.anchors[span] = kept.hi * sum;
            }
            for (int r = 4 * warp; r < da4; r += 4 * WARPS) {                   // four rows of the state, a lane a column
                float u[4] = {};
#pragma unroll 2
                for (int j = 0; j < L; j += 4) {       // (tokens behind the sequence are zeros)
                    const float4 f4 = at4(t.colf + j);
                    const float ff[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float y = ff[q] * t.C[(j + q) * COLS + lane];
                        const float4 x4 = at4(t.B + (j + q) * lda + r);
                        u[0] = fmaf(x4.x, y, u[0]);
                        u[1] = fmaf(x4.y, y, u[1]);
                        u[2] = fmaf(x4.z, y, u[2]);
                        u[3] = fmaf(x4.w, y, u[3]);
                    }
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) S[(r + q) * COLS + lane] = lin::keep(kept, S[(r + q) * COLS + lane], u[q]);
            }
        }
        __syncthreads();
    }
    if (STATE) {
        mix::wait_behind();                            // (the walk before it enters its segments from the same states)
        for (int e = tid; e < da * COLS; e += THREADS) seg_at[e] = S[e];
        if (tid == 0 && blk == 0) w.seg_kept[slot * w.H + h] = all.hi;
    } else if (w.s_out && last) {
        for (int e = tid; e < da * COLS; e += THREADS) {
            const int r = w.s_c == 1 ? e / COLS : e % da, cc = w.s_c == 1 ? e % COLS : e / da;
            if (cc < cols) w.s_out[at_state(r, cc)] = S[r * COLS + cc];
        }
    }
    lin::last_behind();
}

// One block for each (span slot, head), a thread a token: sums of at most kLinSpan terms.
constexpr int DG_WARPS = kLinSpan / 32;
__global__ void __launch_bounds__(kLinSpan) lin_dg_kernel(const LinDg a) {
    __shared__ float plus_s[DG_WARPS], minus_s[DG_WARPS], pairs_s[DG_WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.x % a.H;
    const int64_t slot = blockIdx.x / a.H;
    const int n = lin::slot_sequence(a.cu, a.N(), a.T, kLinSpan, slot);
    int64_t first;
    int len;
    lin::sequence(a.cu, a.T, n, first, len);
    const int64_t at = (slot - (first / kLinSpan + n)) * kLinSpan;
    if (at < 0 || at >= len) {
        if (a.per_head && tid == 0) a.part[slot * a.H + h] = 0.f;
        return;
    }
    const bool in = at + tid < len;
    float plus = 0.f, minus = 0.f, pairs = 0.f;
    if (in) {
        const int64_t t = (int64_t)h * a.rows() + first + at + tid, step = (int64_t)a.H * a.rows();
        for (int k = 0; k < a.blocks; ++k) {
            plus += a.plus[t + k * step];
            minus += a.minus[t + k * step];
        }
        for (int k = 0; k < a.pair_blocks; ++k) pairs += a.pairs[t + k * step] - (a.pairs_minus ? a.pairs_minus[t + k * step] : 0.f);
    }
    float behind = plus, behind_pairs = pairs, before = minus;       // from this token on; up to it
    for (int m = 1; m < 32; m <<= 1) {
        const float x = __shfl_down_sync(0xffffffffu, behind, m), y = __shfl_down_sync(0xffffffffu, behind_pairs, m);
        const float z = __shfl_up_sync(0xffffffffu, before, m);
        if (lane + m < 32) {
            behind += x;
            behind_pairs += y;
        }
        if (lane >= m) before += z;
    }
    if (lane == 0) {
        plus_s[warp] = behind;
        pairs_s[warp] = behind_pairs;
    }
    if (lane == 31) minus_s[warp] = before;
    before = __shfl_up_sync(0xffffffffu, before, 1);
    if (lane == 0) before = 0.f;
    __syncthreads();
    const int per = a.chunk / 32, chunk = warp / per;                // warps of a chunk
    float dg = behind + behind_pairs + before;
    for (int i = warp + 1; i < (chunk + 1) * per; ++i) dg += plus_s[i] + pairs_s[i];
    for (int i = chunk * per; i < warp; ++i) dg += minus_s[i];
    for (int k = 0; k < a.anchor_blocks; ++k) dg += a.anchors[(slot * a.H + h) * a.anchor_blocks + k];
    for (int i = 0; i < chunk * per; ++i) dg += minus_s[i];
    for (int i = per; i < (chunk + 1) * per; ++i) dg -= plus_s[i];
    if (!a.per_head) {
        if (in) a.dg[(first + at + tid) * a.H + h] = dg;
        return;
    }
    float all = in ? dg : 0.f;
    for (int m = 16; m > 0; m >>= 1) all += __shfl_xor_sync(0xffffffffu, all, m);
    __syncthreads();
    if (lane == 0) plus_s[warp] = all;
    __syncthreads();
    if (tid == 0) {
        float t = 0.f;
        for (int i = 0; i < DG_WARPS; ++i) t += plus_s[i];
        a.part[slot * a.H + h] = t;
    }
}

__global__ void lin_dg_sum_kernel(const float* part, float* dg, int64_t slots, int H) {
    const int h = blockIdx.x, lane = threadIdx.x;
    double s = 0.0;
    for (int64_t i = lane; i < slots; i += 32) s += (double)part[i * H + h];
    for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    if (lane == 0) dg[h] = (float)s;
}

// V elements a thread; d is a multiple of V.
template <typename T, int V>
__global__ void __launch_bounds__(256) lin_group_sum_kernel(const float* part, T* out, int64_t heads, int group, int d) {
    const int per = d / V;
    for (int64_t head = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; head < heads; head += (int64_t)gridDim.x * blockDim.y)
        for (int i = threadIdx.x; i < per; i += blockDim.x) {
            const float* p = part + head * group * d + i * V;
            mix::Vec<float, V> s, x;
            s.load(p);
            for (int k = 1; k < group; ++k) {
                x.load(p + (int64_t)k * d);
#pragma unroll
                for (int u = 0; u < V; ++u) s.e[u] += x.e[u];
            }
            mix::Vec<T, V> y;
#pragma unroll
            for (int u = 0; u < V; ++u) y.set(u, s.e[u]);
            y.store(out + head * d + i * V);
        }
}

// The states entering the segments of a sequence, segment after segment in the walk's direction, an element of a block's state
// [da][COLS] a thread.
__global__ void __launch_bounds__(256) lin_generic_segments_kernel(const LinWalk w) {
    const int blocks = (w.dc + COLS - 1) / COLS, elements = w.da * COLS, per = (elements + 255) / 256;
    const int e = blockIdx.x % per * 256 + threadIdx.x;
    const int64_t unit = blockIdx.x / per;
    const int blk = (int)(unit % blocks), h = (int)(unit / blocks % w.H), n = (int)(unit / blocks / w.H);
    int64_t first;
    int len;
    lin::sequence(w.cu, w.T, n, first, len);
    const int size = w.seg_chunks * kLinChunk, segs = lin_segments(len, size);
    const int64_t slot0 = first / size + n;
    const int r = e / COLS, c = blk * COLS + e % COLS;
    const bool in = e < elements, inside = in && c < w.dc;
    const int64_t at = ((int64_t)n * w.H + h) * w.da * w.dc + (int64_t)r * w.s_r + (int64_t)c * w.s_c;
    float s = w.s_in && inside ? w.s_in[at] : 0.f;
    mix::wait_behind();                                   // the segments' own states
    mix::let_next();
    for (int k = 0; k < segs && in; ++k) {                // (the last has none of its own: the walk takes it to the end)
        const int64_t slot = slot0 + (w.rev ? segs - 1 - k : k);
        float* p = w.seg_states + ((slot * w.H + h) * blocks + blk) * (int64_t)elements + e;
        const bool own = k + 1 < segs;
        const float x = own ? *p : 0.f;
        const lin::Keep kept = lin::keep_of({own ? w.seg_kept[slot * w.H + h] : 0.f, 0.f});
        *p = s;
        s = lin::keep(kept, s, x);
    }
    if (w.s_out && segs == 0 && inside) w.s_out[at] = s;  // (no tokens: no walk either)
}

// The same for the tensor-core walk, four columns of a row of a block's state a thread.
__global__ void __launch_bounds__(256) lin_segments_kernel(const LinWalk w) {
    constexpr int PER = 128 * kLinCols / 1024;             // blocks of threads for a state
    const int blocks = (w.dc + kLinCols - 1) / kLinCols;
    const int part = blockIdx.x % PER;
    const int64_t unit = blockIdx.x / PER;
    const int blk = (int)(unit % blocks), h = (int)(unit / blocks % w.H), n = (int)(unit / blocks / w.H);
    int64_t first;
    int len;
    lin::sequence(w.cu, w.T, n, first, len);
    const int size = w.seg_chunks * kLinChunk, segs = lin_segments(len, size);
    const int64_t slot0 = first / size + n;
    const int e = part * 1024 + threadIdx.x * 4, row = e / 4 % 128, c = blk * kLinCols + e / 512 * 4;
    const int64_t at = ((int64_t)n * w.H + h) * w.da * w.dc + (int64_t)row * w.s_r;
    float s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = w.s_in && row < w.da && c + i < w.dc ? w.s_in[at + (int64_t)(c + i) * w.s_c] : 0.f;
    const int64_t step = (int64_t)w.H * blocks * (128 * kLinCols);
    float* p = w.seg_states + ((slot0 * w.H + h) * blocks + blk) * (128 * kLinCols) + e;
    if (w.rev) p += (segs - 1) * step;
    mix::wait_behind();                                   // the segments' own states
    mix::let_next();                                      // (whatever starts now, nothing but this kernel runs before it)
    float4 x = segs > 1 ? *reinterpret_cast<const float4*>(p) : make_float4(0, 0, 0, 0);
    for (int k = 0; k < segs; ++k) {                       // (the last has none of its own: the walk takes it to the end)
        float* next = p + (w.rev ? -step : step);
        const float4 y = k + 2 < segs ? *reinterpret_cast<const float4*>(next) : make_float4(0, 0, 0, 0);
        const lin::Keep kept = lin::keep_of({k + 1 < segs ? w.seg_kept[(slot0 + (w.rev ? segs - 1 - k : k)) * w.H + h] : 0.f, 0.f});
        *reinterpret_cast<float4*>(p) = make_float4(s[0], s[1], s[2], s[3]);
        s[0] = lin::keep(kept, s[0], x.x);
        s[1] = lin::keep(kept, s[1], x.y);
        s[2] = lin::keep(kept, s[2], x.z);
        s[3] = lin::keep(kept, s[3], x.w);
        x = y;
        p = next;
    }
    if (w.s_out && segs == 0)                              // (no tokens: no walk either)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (row < w.da && c + i < w.dc) w.s_out[at + (int64_t)(c + i) * w.s_c] = s[i];
}

}  // namespace

cudaError_t launch_lin_walk_generic(const LinWalk& given, bool behind, cudaStream_t s) {
    LinWalk w = given;
    const int64_t walks = (int64_t)w.H * lin_blocks(w.dc, false);
    const int64_t units = walks * (w.seg_chunks > 0 ? lin_slots(w.rows(), w.N(), w.seg_chunks * kLinChunk) : w.N());
    if (units == 0) return cudaSuccess;
    const size_t smem = sizeof(float) * ((size_t)four(w.da) * COLS + CH * PLD + 2 * generic_tile_floats(w.da));
    auto start = [&](auto kernel, bool early) -> cudaError_t {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        return mix::launch_behind(kernel, dim3((unsigned)units), THREADS, smem, early, s, w);
    };
    if (w.seg_chunks > 0) {
        w.wait_first = 0;
        cudaError_t e = w.bf16 ? start(lin_walk_kernel<bf16, true>, behind) : start(lin_walk_kernel<float, true>, behind);
        if (e != cudaSuccess) return e;
        const int64_t blocks = (int64_t)w.N() * walks * ((w.da * COLS + 255) / 256);
        e = mix::launch_behind(lin_generic_segments_kernel, dim3((unsigned)blocks), 256, 0, true, s, w);
        if (e != cudaSuccess) return e;
        behind = true;
    }
    w.wait_first = behind && (w.spans || w.seg_chunks > 0);
    return w.bf16 ? start(lin_walk_kernel<bf16, false>, behind) : start(lin_walk_kernel<float, false>, behind);
}

cudaError_t launch_lin_dg(const LinDg& a, cudaStream_t s) {
    const int64_t slots = lin_span_slots(a.rows(), a.N());
    lin_dg_kernel<<<(unsigned)(slots * a.H), kLinSpan, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.per_head) return e;
    lin_dg_sum_kernel<<<a.H, 32, 0, s>>>(a.part, a.dg, slots, a.H);
    return cudaGetLastError();
}

cudaError_t launch_lin_group_sum(const float* part, void* out, int bf16_out, int64_t rows, int Hk, int group, int d, cudaStream_t s) {
    const int64_t heads = rows * Hk;
    if (heads == 0) return cudaSuccess;
    auto start = [&](auto kernel, auto* to, int V) {
        int x = 8;
        while (x < 32 && x * V < d) x *= 2;
        const int y = 256 / x;
        const int64_t blocks = (heads + y - 1) / y;
        kernel<<<(unsigned)(blocks < 152 * 64 ? blocks : 152 * 64), dim3(x, y), 0, s>>>(part, to, heads, group, d);
        return cudaGetLastError();
    };
    const bool vec = d % 4 == 0 && (uintptr_t)part % 16 == 0 && (uintptr_t)out % 16 == 0;
    if (bf16_out) return vec ? start(lin_group_sum_kernel<bf16, 4>, static_cast<bf16*>(out), 4) : start(lin_group_sum_kernel<bf16, 1>, static_cast<bf16*>(out), 1);
    return vec ? start(lin_group_sum_kernel<float, 4>, static_cast<float*>(out), 4) : start(lin_group_sum_kernel<float, 1>, static_cast<float*>(out), 1);
}

cudaError_t launch_lin_segments(const LinWalk& w, cudaStream_t s) {
    const int64_t blocks = (int64_t)w.N() * w.H * lin_blocks(w.dc, true) * (128 * kLinCols / 1024);
    return mix::launch_behind(lin_segments_kernel, dim3((unsigned)blocks), 256, 0, true, s, w);
}

}  // namespace gdn
