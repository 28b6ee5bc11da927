// Shared parts of the gated linear recurrence's scans (glr_scan.cu, glr_scan_bwd.cu): the tiling, the input buffer, and
// the carry of a tile from the tiles before it.
//
// A row of T tokens is cut into tiles of 64 tokens x W = LANES * V channels.  A block of 256 threads takes one tile after
// another; LANES threads side by side read V channels each, and so the block has 256 / LANES runs of LANES / 4 consecutive
// tokens, each held in the registers of its threads.  The recurrence over a run of tokens is the map h -> A h + H; a run
// in which a sequence starts (backward: ends) forgets h altogether, which is written A = -1 (decays are never negative),
// so that a state that is not a number stays in its own sequence.
//
// The carry into tile p (in scan order) is, in a fixed association whatever the timing, so that results do not change
// from run to run:
//   the state at the start of its group of kGroup tiles, then the maps of the group's tiles before it, composed first.
// A tile publishes its map as soon as it has it; the last of a group publishes the next group's starting state.  So the
// serial chain of a row is T / (64 kGroup) hops, and each byte of the inputs is read once.  A map is one 8-byte word and a
// state one 4-byte word, which are their own flags: the workspace starts as all ones, which no published word is.
// Blocks take tickets for tiles in scan order, one ahead, to have the next tile's inputs on the way while the carry of the
// current one is worked out.  The smallest tile that is not done is always the current one of its block, so waiting ends;
// waits are bounded all the same.
#pragma once

#include "glr_math.cuh"
#include "mixer.h"
#include "mixer_common.cuh"

namespace gdn {
namespace glr {

constexpr int kThreads = 256;
constexpr int kTile = kGlrTile;                  // checkpoints are tile entries
constexpr int kGroup = 16;
constexpr unsigned kEmpty = 0xffffffffu;
constexpr unsigned long long kWaitNs = 2000000000ull;

struct Residency { cudaError_t error; int blocks; };
Residency residency(const void* kernel, size_t smem);

// Workspace of one scan, set to all ones before the launch.
struct Exchange {
    unsigned* ticket;       // the last ticket taken (all ones: none)
    unsigned* gave_up;      // 0 once a block gave up a wait
    unsigned long long* map;    // [tiles][chains][W]: A in the low half, H in the high half
    unsigned* state;        // [groups][chains][W]
    int tiles, chains, total;
};

struct Layout {
    size_t state_off, bytes;
    int tiles, chains;
};
inline Layout layout(int B, int T, int D, int width) {
    Layout l;
    l.tiles = T > kTile ? (T + kTile - 1) / kTile : 1;
    l.chains = B * ((D + width - 1) / width);
    if (l.tiles == 1) {                          // nothing to exchange
        l.state_off = l.bytes = 0;
        return l;
    }
    const size_t groups = (l.tiles + kGroup - 1) / kGroup, row = (size_t)l.chains * width;
    l.state_off = 256 + l.tiles * row * sizeof(unsigned long long);
    l.bytes = (l.state_off + groups * row * sizeof(unsigned) + 255) / 256 * 256;
    return l;
}
inline Exchange exchange(const Layout& l, void* ws) {
    Exchange x{};
    char* p = static_cast<char*>(ws);
    x.tiles = l.tiles;
    x.chains = l.chains;
    x.total = l.tiles * l.chains;
    if (l.tiles == 1) return x;
    x.ticket = reinterpret_cast<unsigned*>(p);
    x.gave_up = x.ticket + 1;
    x.map = reinterpret_cast<unsigned long long*>(p + 256);
    x.state = reinterpret_cast<unsigned*>(p + l.state_off);
    return x;
}

__device__ __forceinline__ float apply(float A, float H, float h) { return A < 0.f ? H : fmaf(A, h, H); }
__device__ __forceinline__ float both(float A1, float A2) { return A1 < 0.f || A2 < 0.f ? -1.f : A1 * A2; }

__device__ __forceinline__ unsigned long long load_word(const unsigned long long* p) {
    unsigned long long v;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ unsigned load_word(const unsigned* p) {
    unsigned v;
    asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void store_word(unsigned long long* p, unsigned long long v) {
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}
__device__ __forceinline__ void store_word(unsigned* p, unsigned v) {
    asm volatile("st.relaxed.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ unsigned full(float v) {           // a float's bits, which are never kEmpty
    const unsigned b = __float_as_uint(v);
    return b == kEmpty ? 0x7fffffffu : b;
}

// The carry into tile p of a chain, for one channel: called by the W threads that have the channels' maps (A, H) of the
// tile and the state `first` before tile 0 of the row.
__device__ __forceinline__ float carry_in(const Exchange& x, int W, int p, int chain, int ch, float A, float H,
                                          float first, bool publish, unsigned* status) {
    const int group = p / kGroup, start = group * kGroup, n = p - start;
    const bool more = p + 1 < x.tiles, closes = more && n + 1 == kGroup;
    const size_t row = (size_t)x.chains * W, at = (size_t)chain * W + ch;
    if (more && !closes && publish) store_word(x.map + p * row + at, (unsigned long long)full(H) << 32 | full(A));
    if (p == 0) return first;
    unsigned long long m[kGroup - 1];
    unsigned st = group > 0 ? kEmpty : 0u;
#pragma unroll
    for (int j = 0; j < kGroup - 1; ++j) m[j] = j < n ? ~0ull : 0x3f800000ull;       // (the identity: A = 1, H = 0)
    unsigned long long t0 = 0;
    for (int round = 0;; ++round) {
        bool ok = true;
        if (st == kEmpty) st = load_word(x.state + group * row + at);
#pragma unroll
        for (int j = 0; j < kGroup - 1; ++j)
            if ((unsigned)m[j] == kEmpty) m[j] = load_word(x.map + (start + j) * row + at);
#pragma unroll
        for (int j = 0; j < kGroup - 1; ++j) ok = ok && (unsigned)m[j] != kEmpty;
        if (ok && st != kEmpty) break;
        if ((round & 63) == 63) {
            unsigned long long t;
            asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
            if (t0 == 0) t0 = t;
            if (t - t0 > kWaitNs || load_word(x.gave_up) == 0u) {
                store_word(x.gave_up, 0u);
                atomicOr(status, 1u);
                break;                            // the outputs are now unspecified
            }
        }
    }
    float cA = 1.f, cH = 0.f;
#pragma unroll
    for (int j = 0; j < kGroup - 1; ++j) {
        const float a = __uint_as_float((unsigned)m[j]), h = __uint_as_float((unsigned)(m[j] >> 32));
        cH = apply(a, h, cH);
        cA = both(cA, a);
    }
    const float carry = apply(cA, cH, group > 0 ? __uint_as_float(st) : first);
    if (closes && publish) store_word(x.state + (group + 1) * row + at, full(apply(A, H, carry)));
    return carry;
}

struct Channel { float neg_eA, dt; };   // -exp(A_log) (0: g is log a) and dt_bias of a channel
__device__ __forceinline__ Channel channel(const float* A_log, const float* dt_bias, int c) {
    return {A_log ? -expf(A_log[c]) : 0.f, dt_bias ? dt_bias[c] : 0.f};
}

// A block's place in its current tile.
template <int LANES, int V>
struct Place {
    static constexpr int W = LANES * V, kRuns = kThreads / LANES, L = kTile / kRuns;
    int p, chain, b, c0, c, t0;      // tile in the row, chain, batch row, the block's and the thread's first channel,
    int count;                       // the run's first token, and its tokens inside the row
    bool live;                       // the thread's channels exist
    size_t row;                      // the run's first row in [B T]
    __device__ __forceinline__ void set(const Exchange& x, const GlrArgs& a, int id, bool reverse) {
        const int q = id / x.chains, cols = x.chains / a.B;
        chain = id - q * x.chains;
        p = reverse ? x.tiles - 1 - q : q;
        b = chain / cols;
        c0 = (chain - b * cols) * W;
        c = c0 + (int)(threadIdx.x % LANES) * V;
        t0 = p * kTile + (int)(threadIdx.x / LANES) * L;
        live = c < a.D;
        count = min(max(a.T - t0, 0), L);
        row = (size_t)b * a.T + t0;
    }
};

// Packed sequences: which one starts, and which ends, at each token of tile p (-1: none).  Called by threads 0..63.
__device__ __forceinline__ void sequence_marks(const GlrArgs& a, int p, int* starts, int* ends) {
    const int t = p * kTile + threadIdx.x;
    int s = -1, e = -1;
    if (t < a.T) {
        const mix::Span sp = mix::span_of(a.cu, a.n_seqs, a.T, t);
        if (sp.first == t) s = sp.n;
        if (sp.end == t + 1) e = sp.n;
    }
    starts[threadIdx.x] = s;
    ends[threadIdx.x] = e;
}

}  // namespace glr
}  // namespace gdn
