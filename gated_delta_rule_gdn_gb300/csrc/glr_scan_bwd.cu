// Backward of the gated linear recurrence, one pass over the tokens from the last to the first.
//   D_t = dO_t + G_{t+1},  G_t = a_t D_t  (G flows into h_{t-1}; after a sequence's last token it is dhT), and the chain of
//   each token's log a, s and sigma(i) with h_{t-1}.
// A block takes a tile as the forward does.  The states inside it come from the forward's checkpoint at its entry, by
// the same recurrence; G is carried between tiles in reverse (glr_scan.cuh).  So x, g, in_gate and dO are read once and
// the three gradients written once.  The per-channel sums of A_log and dt_bias leave the block as a row of partial sums
// that a second kernel adds in order.
// 470 MB for B4 T4096 D2048 in bf16, 69 us at the copy rate; measured 197 us.  In fp32 279 us (939 MB). Bound by issue: 159 instructions an element
// (8 special functions, two polynomials, five products of stage two) at 2.3 to 2.6 a cycle.  Keeping all seven factors of the
// gradients from stage one, instead of forming them again in stage two, took 314 us: one tile at a time in registers.

#include <type_traits>

#include "glr_scan.cuh"

namespace gdn {
namespace {

using namespace glr;
using mix::bf16;
using mix::Vec;

__device__ unsigned g_glr_bwd_status;   // bit 0: a block gave up a bounded wait

struct BwdSpace { void* scan; float* part; };

// Stage one keeps the decay, 1 - a^2, log a and the input u of a tile's elements in registers; its raw inputs
// stay in shared memory until stage two, which first runs the gradient D through the run from behind, then the state from
// the front, and forms each token's gradients on the way.
constexpr int kBuffers = 3;

template <typename Tx, typename Tg, typename S, bool PACKED>
__global__ void __launch_bounds__(S::kBlock, 2)
glr_bwd_kernel(const GlrArgs a, const Exchange x, float* part) {
    constexpr int LANES = S::LANES, V = S::V, W = S::W, R = S::R, L = S::L, kThreads = S::kThreads;
    static_assert(2 * W <= kCarryThreads, "a carry thread for every channel and direction");
    extern __shared__ __align__(16) unsigned char s_raw[];
    __shared__ float sA[2][R][W], sH[2][R][W], sG[2][R][W], s_sum[3][2][R][W];
    __shared__ unsigned char s_any[2][R];        // bit 0: a sequence starts in the run; bit 1: one ends
    __shared__ int s_start[PACKED ? kPlaces : 1][kTile], s_end[PACKED ? kPlaces : 1][kTile];
    __shared__ bool s_marked[kPlaces][2];        // whether either half of a tile's tokens has a mark
    __shared__ __align__(16) Channel s_chan[kPlaces][W];
    __shared__ Tile s_tile[kPlaces];
    const int tid = threadIdx.x;
    mix::wait_behind();                          // for the clearing
    mix::let_next();
    const auto marked = [&](int i) { return PACKED && (s_marked[i % kPlaces][0] || s_marked[i % kPlaces][1]); };

    if (tid >= kThreads) {                       // the carry threads: the gradient's, the state's
        const int ch = (tid - kThreads) % W, side = (tid - kThreads) / W;
        const auto prepare = [&](int slot) {      // a place's channels and marks
            if (s_tile[slot].chain < 0) return;
            const int pc = tid - kThreads, c = s_tile[slot].c0 + pc;
            if (a.A_log && pc < W && c < a.D) s_chan[slot][pc] = channel(a.A_log, a.dt_bias, c);
            if (!PACKED) return;
            const bool any = sequence_marks(a, s_tile[slot].p, tid - kThreads, s_start[slot], s_end[slot]);
            if (tid % 32 == 0) s_marked[slot][(tid - kThreads) / 32] = any;
        };
        Tickets tickets(x);
        unsigned ticket = 0;
        first_tiles(x, a, W, true, tickets, s_tile, tid == kThreads, [] { __syncthreads(); });
        if (tid == kThreads) ticket = tickets.take();
        __syncwarp();
        S::sync(kMaps);
        for (int i = 0; i < 3; ++i) prepare(i);
        __syncthreads();
        // the sums of tile i over its runs, in order
        const auto sums = [&](int i) {
            const Tile t = s_tile[i % kPlaces];
            if (side > 1 || t.c0 + ch >= a.D) return;
            float s = 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r) s += s_sum[i % 3][side][r][ch];
            const size_t rows = (size_t)a.B * x.tiles, r = (size_t)t.b * x.tiles + t.p;
            part[((side ? rows : 0) + r) * a.D + t.c0 + ch] = s;
        };
        int i = 0;
        for (; s_tile[i % kPlaces].chain >= 0; ++i) {
            const Tile t = s_tile[i % kPlaces];
            const int k = i & 1, ahead = (i + 3) % kPlaces, q = x.tiles - 1 - t.p;
            if (tid == kThreads) {
                s_tile[ahead] = tile_of(x, a, W, ticket, true);
                ticket = tickets.take();
            }
            // what enters the tile: the state from its checkpoint, the gradient behind the row's last token
            const bool live = t.c0 + ch < a.D;
            float enter = 0.f;
            if (side == 0) {
                if (!PACKED && q < kSpan && a.dhT && live) enter = a.dhT[(size_t)t.b * a.D + t.c0 + ch];
            } else if (side == 1 && live && t.p * kTile < a.T) {
                if (t.p > 0 || PACKED) enter = a.ckpt[((size_t)t.b * x.tiles + t.p) * a.D + t.c0 + ch];
                else if (a.h0) enter = a.h0[(size_t)t.b * a.D + t.c0 + ch];
            }
            S::sync(kMaps + k);
            // (a tile without marks forgets nothing inside)
            const auto work = [&](auto marks) {
                constexpr bool M = decltype(marks)::value;
                if (side == 0) {
                    const auto run_A = [&](int r) { return M && (s_any[k][r] & 2) ? -1.f : sA[k][r][ch]; };
                    float A = 1.f, G = 0.f;
#pragma unroll
                    for (int r = R - 1; r >= 0; --r) {
                        G = apply<M>(run_A(r), sG[k][r][ch], G);
                        A = both<M>(A, run_A(r));
                    }
                    float g = carry_in<PACKED>(x, W, q, t.chain, ch, A, G, enter, true, &g_glr_bwd_status);
#pragma unroll
                    for (int r = R - 1; r >= 0; --r) {
                        const float rG = sG[k][r][ch];
                        sG[k][r][ch] = g;
                        g = apply<M>(run_A(r), rG, g);
                    }
                } else if (side == 1) {
                    float h = enter;
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float rA = M && (s_any[k][r] & 1) ? -1.f : sA[k][r][ch], rH = sH[k][r][ch];
                        sH[k][r][ch] = h;
                        h = apply<M>(rA, rH, h);
                    }
                }
            };
            if (marked(i)) work(std::bool_constant<PACKED>{}); else work(std::false_type{});
            S::arrive(kCarry + k);
            if (a.dA && i >= 2) sums(i - 2);     // (stage two of tile i - 2 came before the maps of tile i)
            prepare(ahead);
        }
        if (a.dA && i > 0) {
            S::sync(kMaps + (i & 1));           // the compute threads are through
            if (i >= 2) sums(i - 2);
            sums(i - 1);
        }
        return;
    }

    // the compute threads
    const int run = tid / LANES, lane = tid % LANES, arrays = a.gi ? 4 : 3;
    const int bytes = L * kThreads * (int)(sizeof(Vec<Tg, V>) + (arrays - 1) * sizeof(Vec<Tx, V>));
    const auto buf_g = [&](int i) { return reinterpret_cast<Vec<Tg, V>*>(s_raw + i % kBuffers * bytes) + tid; };
    const auto buf_x = [&](int i) {              // x, dO, and the input gate's logits: [L][kThreads] each
        return reinterpret_cast<Vec<Tx, V>*>(s_raw + i % kBuffers * bytes + L * kThreads * sizeof(Vec<Tg, V>)) + tid;
    };
    const auto fetch = [&](int i) {
        const Tile t = s_tile[i % kPlaces];
        const int c = t.c0 + lane * V, t0 = t.p * kTile + run * L;
        const int n = t.chain >= 0 && c < a.D ? min(a.T - t0, L) : 0;
        const size_t row = (size_t)t.b * a.T + t0;
        const Tg* g = static_cast<const Tg*>(a.g) + row * a.ldg + c;
        const Tx* xp = static_cast<const Tx*>(a.x) + row * a.ldx + c;
        const Tx* ip = static_cast<const Tx*>(a.gi) + row * a.ldi + c;
        const Tx* op = static_cast<const Tx*>(a.dO) + row * a.D + c;
        Vec<Tg, V>* bg = buf_g(i);
        Vec<Tx, V>* bx = buf_x(i);
        if (n == L) {
#pragma unroll
            for (int j = 0; j < L; ++j) {
                mix::copy_async(bg + j * kThreads, g, true);
                mix::copy_async(bx + j * kThreads, xp, true);
                mix::copy_async(bx + (L + j) * kThreads, op, true);
                if (a.gi) mix::copy_async(bx + (2 * L + j) * kThreads, ip, true);
                op += a.D;
                g += a.ldg;
                xp += a.ldx;
                ip += a.ldi;
            }
            mix::copies_close();
            return;
        }
#pragma unroll 1
        for (int j = 0; j < L; ++j) {            // the row's end, or no channels
            mix::copy_async(bg + j * kThreads, j < n ? g : static_cast<const Tg*>(a.g), j < n);
            mix::copy_async(bx + j * kThreads, j < n ? xp : static_cast<const Tx*>(a.x), j < n);
            mix::copy_async(bx + (L + j) * kThreads, j < n ? op : static_cast<const Tx*>(a.dO), j < n);
            if (a.gi) mix::copy_async(bx + (2 * L + j) * kThreads, j < n ? ip : static_cast<const Tx*>(a.gi), j < n);
            g += a.ldg;
            xp += a.ldx;
            ip += a.ldi;
            op += a.D;
        }
        mix::copies_close();
    };
    struct Held { float al[L][V], power[L][V], la[L][V], u[L][V]; };
    const auto marks = [&](int i, unsigned* starts, unsigned* ends) {
        *starts = *ends = 0;
#pragma unroll
        for (int j = 0; j < L; ++j) {
            *starts |= (s_start[i % kPlaces][run * L + j] >= 0 ? 1u : 0u) << j;
            *ends |= (s_end[i % kPlaces][run * L + j] >= 0 ? 1u : 0u) << j;
        }
    };
    // dO, with what enters behind a sequence's last token
    const auto grad_o = [&](int i, int j, int c, bool end, float (&d)[V]) {
        const Vec<Tx, V> o = buf_x(i)[(L + j) * kThreads];
#pragma unroll
        for (int v = 0; v < V; ++v) d[v] = o.get(v);
        if (end && a.dhT && c < a.D)
#pragma unroll
            for (int v = 0; v < V; ++v) d[v] += a.dhT[(size_t)s_end[i % kPlaces][run * L + j] * a.D + c + v];
    };

    // stage one: decays and inputs of the run, and its maps: (A, H) of the state, (A, G) of the gradient
    const auto maps = [&](int i, Held& q, auto marks_here) {
        constexpr bool M = decltype(marks_here)::value;
        const Tile t = s_tile[i % kPlaces];
        const int c = t.c0 + lane * V, count = a.T - (t.p * kTile + run * L);
        const bool live = c < a.D;
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const Vec<Tg, V> g = buf_g(i)[j * kThreads];
            const Vec<Tx, V> xv = buf_x(i)[j * kThreads];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                q.la[j][v] = g.get(v);
                q.u[j][v] = xv.get(v);
            }
        }
        if (a.gi) {
#pragma unroll
            for (int j = 0; j < L; ++j) {
                const Vec<Tx, V> gi = buf_x(i)[(2 * L + j) * kThreads];
#pragma unroll
                for (int v = 0; v < V; ++v) q.u[j][v] *= sigmoid(gi.get(v));
            }
        }
        log_decays<L, V>(a, s_chan[i % kPlaces] + lane * V, q.la);
        decays<L, V>(q.la, [&](int j, int v, const auto&... d) {
            if (a.normalize) {
                input_powers(&q.power[j][v], d...);
                times_factors<sizeof...(d)>(&q.u[j][v], &q.power[j][v]);
            }
            ((q.al[j][v++] = d.a), ...);
        });
        if (count < L) {                         // past the row's end state and gradient stay
#pragma unroll
            for (int j = 0; j < L; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) q.al[j][v] = j < count ? q.al[j][v] : 1.f;
        }
        unsigned starts = 0, ends = 0;
        if (M) marks(i, &starts, &ends);
        float A[V], H[V], G[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            A[v] = 1.f;
            H[v] = G[v] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const bool start = M && ((starts >> j) & 1);
            if (start && a.h0 && live)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    q.u[j][v] = fmaf(q.al[j][v], a.h0[(size_t)s_start[i % kPlaces][run * L + j] * a.D + c + v], q.u[j][v]);
            if (start) {
#pragma unroll
                for (int v = 0; v < V; ++v) H[v] = q.u[j][v];
            } else {
                mix::fma_row(H, q.al[j], H, q.u[j]);
            }
            mix::mul_row(A, A, q.al[j]);
        }
#pragma unroll
        for (int j = L - 1; j >= 0; --j) {
            const bool end = M && ((ends >> j) & 1);
            float d[V];
            grad_o(i, j, c, end, d);
            if (!end) mix::add_row(d, d, G);
            mix::mul_row(G, q.al[j], d);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            sA[i & 1][run][lane * V + v] = A[v];
            sH[i & 1][run][lane * V + v] = H[v];
            sG[i & 1][run][lane * V + v] = G[v];
        }
        if (PACKED && lane == 0) s_any[i & 1][run] = (starts ? 1 : 0) | (ends ? 2 : 0);
        S::arrive(kMaps + (i & 1));
    };

    // stage two: with h_{t-1}, and D the gradient of h_t,
    //   dx = D s sigma(i), di = dx x (1 - sigma(i)), dla = D (a h_{t-1} - sigma(i) x a^2 / s), dg = dla dlog a/dg
    const auto gradients = [&](int i, const Held& q, auto marks_here) {
        constexpr bool M = decltype(marks_here)::value;
        const Tile t = s_tile[i % kPlaces];
        const int c = t.c0 + lane * V, t0 = t.p * kTile + run * L;
        const bool live = c < a.D;
        const int n = live ? a.T - t0 : 0;
        unsigned starts = 0, ends = 0;
        if (M) marks(i, &starts, &ends);
        float D[L][V], G[V], h[V], pA[V], pdt[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            G[v] = sG[i & 1][run][lane * V + v];
            h[v] = sH[i & 1][run][lane * V + v];
            pA[v] = pdt[v] = 0.f;
        }
#pragma unroll
        for (int j = L - 1; j >= 0; --j) {
            const bool end = M && ((ends >> j) & 1);
            grad_o(i, j, c, end, D[j]);
            if (!end) mix::add_row(D[j], D[j], G);
            mix::mul_row(G, q.al[j], D[j]);
            if (M && a.dh0 && live) {
                const int s = s_start[i % kPlaces][run * L + j];
                if (s >= 0)
#pragma unroll
                    for (int v = 0; v < V; ++v) a.dh0[(size_t)s * a.D + c + v] = G[v];
            }
        }
        Channel ch[V];
#pragma unroll
        for (int v = 0; v < V; ++v) ch[v] = s_chan[i % kPlaces][lane * V + v];
        const size_t at = ((size_t)t.b * a.T + t0) * a.D + c;
        Tx* dx_p = static_cast<Tx*>(a.dx) + at;
        Tx* di_p = static_cast<Tx*>(a.di) + at;
        Tg* dg_p = static_cast<Tg*>(a.dg) + at;
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const bool start = M && ((starts >> j) & 1);
            float hp[V];
#pragma unroll
            for (int v = 0; v < V; ++v) hp[v] = h[v];
            if (!start) {
                mix::fma_row(h, q.al[j], h, q.u[j]);
            } else
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    h[v] = q.u[j][v];
                    hp[v] = a.h0 && live ? a.h0[(size_t)s_start[i % kPlaces][run * L + j] * a.D + c + v] : 0.f;
                }
            const Vec<Tx, V> xv = buf_x(i)[j * kThreads];
            float w[V], y[V], xs[V], dla[V], dz[V];   // s sigma(i), x (1 - sigma(i)), x sigma(i)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                xs[v] = xv.get(v);
                w[v] = 1.f;
                y[v] = 0.f;
            }
            if (a.gi) {
                const Vec<Tx, V> gi = buf_x(i)[(2 * L + j) * kThreads];
                float f[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    // 1 - sigma(i) = exp(-i) sigma(i), with exp(-i) kept finite for that product: a shut gate's sigma is 0
                    // here as it is forward, whatever the input behind it
                    const float e = ex2(gi.get(v) * -kLog2e);
                    w[v] = rcp(1.f + e);
                    f[v] = fminf(e, 3.402823466e38f);
                }
                mix::mul_row(xs, xs, w);
                mix::mul_row(y, xs, f);
            }
            mix::mul_row(dla, q.al[j], hp);
            if (a.normalize) {
                float s[V], m[V], sq[V], down[V], up[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    // ds/dlog a = -a^2 / s, taken as 0 where s = 0 (log a = 0: the derivative does not exist there)
                    m[v] = q.power[j][v] > 0.f ? rsq(q.power[j][v]) : 0.f;
                    down[v] = 1.f / kFactor;
                    up[v] = -kFactor;
                }
                mix::mul_row(s, q.power[j], m);
                mix::mul_row(s, s, down);
                mix::mul_row(m, m, up);
                mix::mul_row(w, w, s);
                mix::mul_row(m, m, xs);
                mix::mul_row(sq, q.al[j], q.al[j]);
                mix::fma_row(dla, m, sq, dla);
            }
            mix::mul_row(dla, dla, D[j]);
#pragma unroll
            for (int v = 0; v < V; ++v) dz[v] = dla[v];
            if (a.A_log) {
                const Vec<Tg, V> g = buf_g(i)[j * kThreads];
                float t[V], z[V], ez[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    z[v] = g.get(v) + ch[v].dt;
                    ez[v] = tail_root(z[v]);
                }
                mix::mul_row(ez, ez, ez);
#pragma unroll
                for (int v = 0; v < V; ++v) t[v] = ch[v].neg_eA * sigmoid(z[v], ez[v]);
                mix::mul_row(dz, dz, t);
                if (j < n) {
                    mix::fma_row(pA, dla, q.la[j], pA);
                    mix::add_row(pdt, pdt, dz);
                }
            }
            float dw[V], dy[V];
            mix::mul_row(dw, D[j], w);
            mix::mul_row(dy, dw, y);
            Vec<Tx, V> dx, di;
            Vec<Tg, V> dg;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                dx.set(v, dw[v]);
                di.set(v, dy[v]);
                dg.set(v, dz[v]);
            }
            if (j < n) {
                dx.store(dx_p);
                dg.store(dg_p);
                if (a.gi) di.store(di_p);
            }
            dx_p += a.D;
            di_p += a.D;
            dg_p += a.D;
        }
        if (!PACKED && a.dh0 && live && t.p == 0 && run == 0)
#pragma unroll
            for (int v = 0; v < V; ++v) a.dh0[(size_t)t.b * a.D + c + v] = G[v];
        if (PACKED && a.dh0 && live) {
            // empty sequences: what enters behind leaves in front; the row's tiles share them
            for (int s = t.p * R + run; s < a.n_seqs; s += x.tiles * R) {
                if (mix::clamp_off(a.cu[s + 1], a.T) > mix::clamp_off(a.cu[s], a.T)) continue;
#pragma unroll
                for (int v = 0; v < V; ++v) a.dh0[(size_t)s * a.D + c + v] = a.dhT ? a.dhT[(size_t)s * a.D + c + v] : 0.f;
            }
        }
        if (a.dA)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s_sum[i % 3][0][run][lane * V + v] = pA[v];
                s_sum[i % 3][1][run][lane * V + v] = pdt[v];
            }
    };

    __syncthreads();
    fetch(0);
    S::arrive(kMaps);
    __syncthreads();
    if (s_tile[0].chain < 0) return;
    fetch(1);
    Held q, before;                              // the current tile's, and the one's before it
    for (int i = 0;; ++i) {
        const bool more = s_tile[i % kPlaces].chain >= 0;
        if (more) {
            mix::copies_wait<1>();
            if (marked(i)) maps(i, q, std::bool_constant<PACKED>{}); else maps(i, q, std::false_type{});
        }
        if (i > 0) {
            S::sync(kCarry + ((i - 1) & 1));
            if (marked(i - 1)) gradients(i - 1, before, std::bool_constant<PACKED>{});
            else gradients(i - 1, before, std::false_type{});
        }
        if (!more) {
            if (a.dA) S::arrive(kMaps + (i & 1));
            break;
        }
        fetch(i + 2);                            // (into the buffer of tile i - 1)
        before = q;
    }
}

// column sums of part [2][rows][D]: 32 channels a block, 8 row lanes, joined in order
__global__ void __launch_bounds__(256) glr_param_kernel(const float* part, int rows, int D, float* dA, float* ddt) {
    __shared__ float s[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    const float* src = part + (size_t)blockIdx.y * rows * D;
    float* out = blockIdx.y ? ddt : dA;
    if (!out) return;
    mix::wait_behind();
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

template <typename Tx, typename Tg, typename S, bool PACKED>
cudaError_t bwd(const GlrArgs& a, const BwdSpace& sp, cudaStream_t s) {
    const Layout l = layout(a.B, a.T, a.D, S::W);
    const Exchange x = exchange(l, sp.scan);
    if (l.bytes) {
        const cudaError_t e = clear(sp.scan, l.bytes, s);
        if (e != cudaSuccess) return e;
    }
    const auto kernel = glr_bwd_kernel<Tx, Tg, S, PACKED>;
    const int smem = kBuffers * S::L * S::kThreads * S::V * (int)(sizeof(Tg) + (a.gi ? 3 : 2) * sizeof(Tx));
    static Residency res[2];                     // without and with the input gate
    int blocks = 0;
    cudaError_t e = res[a.gi != nullptr].get(reinterpret_cast<const void*>(kernel), S::kBlock, smem, &blocks);
    if (e != cudaSuccess) return e;
    e = mix::launch_behind(kernel, x.total < blocks ? x.total : blocks, S::kBlock, smem, l.bytes > 0, s, a, x, sp.part);
    if (e != cudaSuccess || !a.dA) return e;
    return mix::launch_behind(glr_param_kernel, dim3((a.D + 31) / 32, 2), 256, 0, true, s, sp.part, a.B * l.tiles, a.D, a.dA,
                              a.ddt);
}

template <typename Tx, typename Tg, typename S>
cudaError_t bwd_packed(const GlrArgs& a, const BwdSpace& sp, cudaStream_t s) {
    return a.cu ? bwd<Tx, Tg, S, true>(a, sp, s) : bwd<Tx, Tg, S, false>(a, sp, s);
}

template <typename Tx, typename Tg>
cudaError_t bwd_wide(const GlrArgs& a, const BwdSpace& sp, cudaStream_t s) {
    if (glr_vector(a, 2)) return bwd_packed<Tx, Tg, Shape<16, 2, 4>>(a, sp, s);
    return bwd_packed<Tx, Tg, Shape<32, 1, 8>>(a, sp, s);
}

// The backward's workspace: the scan's exchange, the partial sums of the parameters, and the checkpoints that the
// caller did not keep (with the forward's exchange for computing them in the scan's place).
size_t up(size_t v) { return (v + 255) / 256 * 256; }
int tiles_of(const GlrArgs& a) { return layout(a.B, a.T, a.D, 32).tiles; }
size_t part_bytes(const GlrArgs& a) { return up(2 * (size_t)a.B * tiles_of(a) * a.D * sizeof(float)); }

}  // namespace

size_t glr_workspace_bytes(const GlrArgs& a, bool backward) {
    size_t scan = 0;
    for (int width = 32; width <= 64; width *= 2) {
        const size_t n = layout(a.B, a.T, a.D, width).bytes;
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
