// Shared parts of the gated linear recurrence's scans (glr_scan.cu, glr_scan_bwd.cu): the tiling, the input buffer, and
// the carry of a tile from the tiles before it.
//
// A row of T tokens is cut into tiles of 64 tokens x W = LANES * V channels.  A block takes one tile after another; LANES
// threads side by side read V channels each and L consecutive tokens, a run, and 64 / L such rows of threads take the
// tile.  The recurrence over a run of tokens is the map h -> A h + H; a run in which a sequence starts (backward: ends)
// forgets h altogether, which is written A = -1 (decays are never negative), so that a state that is not a number stays in
// its own sequence.
//
// The carry into tile p (in scan order) is, in a fixed association whatever the timing, so that results do not change
// from run to run: the state at the start of its block of 64 tiles, then the maps of the block's groups of 8 tiles before
// its own, then the maps of its group's tiles before it.  A tile publishes its map as soon as it has it; the last of a
// group the group's map as soon as it has the other seven; the last of a block the next block's starting state.  So the
// serial chain of a row is T / 4096 hops, a carry takes in at most 14 maps, and each byte of the inputs is read once.  A map
// is one 8-byte word and a state one 4-byte word, which are their own flags: the workspace starts as all ones, which no
// published word is.
// Blocks take tickets for tiles in scan order, a few ahead, and go through their tiles in that order.  All that the smallest
// tile without a carry waits for is therefore done or under way, and waiting ends; waits are bounded all the same.
#pragma once

#include "glr_math.cuh"
#include "mixer.h"
#include "mixer_common.cuh"
#include "residency.h"

namespace gdn {
namespace glr {

constexpr int kTile = kGlrTile;                  // checkpoints are tile entries
constexpr int kGroup = 8, kSpan = kGroup * kGroup;      // tiles a group, and a block of groups
constexpr unsigned kEmpty = 0xffffffffu;
constexpr unsigned long long kWaitNs = 2000000000ull;

// A scan is launched behind the clearing of its workspace (mix::launch_behind).  The clearing starts after all earlier
// work of the stream; the scan's blocks start while it runs, and touch memory only after their wait for it (against a memset
// before the scan: 1000 tokens x 2048 channels 14.7 us and 17.5, B4 T4096 D2048 86 and 89 forward, 199 and 203 backward,
// 65,536 packed tokens x 4096 channels 763 and 755 forward, 1613 and 1619 backward).
cudaError_t clear(void* ws, size_t bytes, cudaStream_t s);       // bytes in steps of 256, ws on a 256-byte boundary

// Workspace of one scan, set to all ones before the launch.
struct Exchange {
    unsigned* ticket;       // the last ticket taken (all ones: none)
    unsigned* gave_up;      // 0 once a block gave up a wait
    unsigned long long* map;        // [tiles][chains][W]: A in the low half, H in the high half
    unsigned long long* group_map;  // [groups][chains][W]
    unsigned* state;                // [blocks of groups][chains][W]
    int tiles, chains, total;
};

struct Layout {
    size_t group_off, state_off, bytes;
    int tiles, chains;
};
inline Layout layout(int B, int T, int D, int width) {
    Layout l;
    l.tiles = T > kTile ? (T + kTile - 1) / kTile : 1;
    l.chains = B * ((D + width - 1) / width);
    if (l.tiles == 1) {                          // nothing to exchange
        l.group_off = l.state_off = l.bytes = 0;
        return l;
    }
    const size_t groups = (l.tiles + kGroup - 1) / kGroup, spans = (l.tiles + kSpan - 1) / kSpan;
    const size_t row = (size_t)l.chains * width;
    l.group_off = 256 + l.tiles * row * sizeof(unsigned long long);
    l.state_off = l.group_off + groups * row * sizeof(unsigned long long);
    l.bytes = (l.state_off + spans * row * sizeof(unsigned) + 255) / 256 * 256;
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
    x.group_map = reinterpret_cast<unsigned long long*>(p + l.group_off);
    x.state = reinterpret_cast<unsigned*>(p + l.state_off);
    return x;
}

// Maps applied and composed; without packed sequences none forgets.
template <bool PACKED>
__device__ __forceinline__ float apply(float A, float H, float h) { return PACKED && A < 0.f ? H : fmaf(A, h, H); }
template <bool PACKED>
__device__ __forceinline__ float both(float A1, float A2) {
    return PACKED && (A1 < 0.f || A2 < 0.f) ? -1.f : A1 * A2;
}

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

__device__ __forceinline__ unsigned long long word_of(float A, float H) { return (unsigned long long)full(H) << 32 | full(A); }
constexpr unsigned long long kIdentity = 0x3f800000ull;       // A = 1, H = 0

// Load those of the first n (<= 7) words of a column that are still empty; whether all are there now.
__device__ __forceinline__ bool gather(unsigned long long (&m)[kGroup - 1], const unsigned long long* p, size_t step) {
#pragma unroll
    for (int j = 0; j < kGroup - 1; ++j)
        if ((unsigned)m[j] == kEmpty) m[j] = load_word(p + j * step);
    bool ok = true;
#pragma unroll
    for (int j = 0; j < kGroup - 1; ++j) ok = ok && (unsigned)m[j] != kEmpty;
    return ok;
}
template <bool PACKED>
__device__ __forceinline__ void compose(const unsigned long long (&m)[kGroup - 1], float& A, float& H) {
    A = 1.f;
    H = 0.f;
#pragma unroll
    for (int j = 0; j < kGroup - 1; ++j) {
        const float a = __uint_as_float((unsigned)m[j]);
        H = apply<PACKED>(a, __uint_as_float((unsigned)(m[j] >> 32)), H);
        A = both<PACKED>(A, a);
    }
}

// Time out of a wait, looked at once in 64 rounds: true if the block gives up (its outputs are then unspecified).
struct Patience {
    unsigned long long t0 = 0;
    int round = 0;
    __device__ __forceinline__ bool over(const Exchange& x, unsigned* status) {
        if ((++round & 63) != 0) return false;
        unsigned long long t;
        asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
        if (t0 == 0) t0 = t;
        if (t - t0 <= kWaitNs && load_word(x.gave_up) != 0u) return false;
        store_word(x.gave_up, 0u);
        atomicOr(status, 1u);
        return true;
    }
};

// Hand over the map (A, H) of tile p of a chain, for one channel, and get the carry into it; `first` is the state before
// tile 0 of the row.
template <bool PACKED>
__device__ __forceinline__ float carry_in(const Exchange& x, int W, int p, int chain, int ch, float A, float H, float first,
                                          bool publish, unsigned* status) {
    const size_t row = (size_t)x.chains * W, at = (size_t)chain * W + ch;
    const int in_group = p % kGroup, group = p / kGroup, in_span = group % kGroup, span = p / kSpan;
    const bool more = p + 1 < x.tiles, last = in_group == kGroup - 1;
    if (more && !last && publish) store_word(x.map + p * row + at, word_of(A, H));
    unsigned long long m[kGroup - 1], g[kGroup - 1];
#pragma unroll
    for (int j = 0; j < kGroup - 1; ++j) {
        m[j] = j < in_group ? ~0ull : kIdentity;
        g[j] = j < in_span ? ~0ull : kIdentity;
    }
    const unsigned long long* mp = x.map + (size_t)(p - in_group) * row + at;
    const unsigned long long* gp = x.group_map + (size_t)(group - in_span) * row + at;
    unsigned st = span > 0 ? load_word(x.state + span * row + at) : 0u;
    gather(g, gp, row);
    Patience wait;
    while (!gather(m, mp, row))
        if (wait.over(x, status)) break;
    float mA, mH;
    compose<PACKED>(m, mA, mH);
    if (more && last && in_span != kGroup - 1)
        store_word(x.group_map + (size_t)group * row + at, word_of(both<PACKED>(mA, A), apply<PACKED>(A, H, mH)));
    while (!gather(g, gp, row) || st == kEmpty) {
        if (st == kEmpty) st = load_word(x.state + span * row + at);
        if (wait.over(x, status)) break;
    }
    float gA, gH;
    compose<PACKED>(g, gA, gH);
    const float carry = apply<PACKED>(mA, mH, apply<PACKED>(gA, gH, span > 0 ? __uint_as_float(st) : first));
    if (more && p % kSpan == kSpan - 1) store_word(x.state + (size_t)(span + 1) * row + at, full(apply<PACKED>(A, H, carry)));
    return carry;
}

struct Channel { float neg_eA, dt; };   // -exp(A_log) (0: g is log a) and dt_bias of a channel
__device__ __forceinline__ Channel channel(const float* A_log, const float* dt_bias, int c) {
    return {A_log ? -expf(A_log[c]) : 0.f, dt_bias ? dt_bias[c] : 0.f};
}

// log a of a run's gates, in place; `chan` the parameters of its channels.
template <int L, int V>
__device__ __forceinline__ void log_decays(const GlrArgs& a, const Channel* chan, float (&la)[L][V]) {
    if (a.A_log) {
        Channel ch[V];
#pragma unroll
        for (int v = 0; v < V; ++v) ch[v] = chan[v];
#pragma unroll
        for (int j = 0; j < L; ++j) {
            if constexpr (V % 2 == 0) {
#pragma unroll
                for (int v = 0; v < V; v += 2)
                    softplus(la[j][v] + ch[v].dt, la[j][v + 1] + ch[v + 1].dt, ch[v].neg_eA, ch[v + 1].neg_eA, la[j][v], la[j][v + 1]);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float z = la[j][v] + ch[v].dt;
                    la[j][v] = ch[v].neg_eA * softplus(z, tail(z));
                }
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < L; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) la[j][v] = min_nan(la[j][v], 88.f);
    }
}
// f(j, v, decay of element v, of element v + 1) for every pair of a run, or f(j, v, decay) for every element if V is odd.
template <int L, int V, typename F>
__device__ __forceinline__ void decays(float (&la)[L][V], F f) {
#pragma unroll
    for (int j = 0; j < L; ++j) {
        if constexpr (V % 2 == 0) {
#pragma unroll
            for (int v = 0; v < V; v += 2) {
                Decay d0, d1;
                decay(la[j][v], la[j][v + 1], d0, d1);
                f(j, v, d0, d1);
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) f(j, v, decay(la[j][v]));
        }
    }
}

// The block's division of work.  Its compute threads take a tile in two stages: the maps of their runs (stage one), and
// with the states that enter the runs the outputs (stage two).  Stage two of a tile comes after stage one of the next, so
// that the carry, which kCarryThreads threads of their own work out in between, has that long to arrive.  Two more
// tiles' inputs are on the way meanwhile.  Per tile i the two sides meet at two barriers, each of one parity of i:
//   MAPS   the compute threads have left their runs' maps in shared memory;
//   CARRY  the carry threads have left the runs' entering states there, and tile i + 3's place in the ring of places.
// (Its channels' parameters and sequence marks follow, in time for CARRY of tile i + 1.)
constexpr int kCarryThreads = 64, kPlaces = 8;
constexpr int kMaps = 1, kCarry = 3;

template <int LANES_, int V_, int L_>
struct Shape {
    static constexpr int LANES = LANES_, V = V_, L = L_, W = LANES * V, R = kTile / L;
    static constexpr int kThreads = LANES * R, kBlock = kThreads + kCarryThreads;      // compute threads, all threads
    static __device__ __forceinline__ void arrive(int id) {
        asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(kBlock) : "memory");
    }
    static __device__ __forceinline__ void sync(int id) {
        asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(kBlock) : "memory");
    }
};

// A tile: its place in the row, batch row, first channel and chain (chain < 0: there is none).
struct Tile { int p, b, c0, chain; };
__device__ __forceinline__ Tile tile_of(const Exchange& x, const GlrArgs& a, int W, unsigned id, bool reverse) {
    if (id >= (unsigned)x.total) return {0, 0, 0, -1};
    const int q = id / x.chains, chain = id - q * x.chains, cols = x.chains / a.B, b = chain / cols;
    return {reverse ? x.tiles - 1 - q : q, b, (chain - b * cols) * W, chain};
}
// Rows with a single tile need no tickets: blocks stride over the chains.
struct Tickets {
    unsigned* counter;
    unsigned next;
    __device__ __forceinline__ explicit Tickets(const Exchange& x) : counter(x.ticket), next(blockIdx.x) {}
    __device__ __forceinline__ unsigned take() {
        if (counter) return atomicAdd(counter, 1u) + 1u;
        const unsigned t = next;
        next += gridDim.x;
        return t;
    }
};
// A block's first three tiles, one ticket after the other, so that every block has its first before any has its second:
// blocks that take several at once have neighbouring tiles at different places in their queues, and wait for each other's
// queues (65,536 tokens x 250 channels: 1.2 ms with three at once, 87 us so; 73 us with what came after).
template <typename Meet>
__device__ __forceinline__ void first_tiles(const Exchange& x, const GlrArgs& a, int W, bool reverse, Tickets& tickets,
                                            Tile* tile, bool leader, Meet meet) {
    if (leader) tile[0] = tile_of(x, a, W, tickets.take(), reverse);
    meet();
    if (leader)
        for (int i = 1; i < 3; ++i) tile[i] = tile_of(x, a, W, tickets.take(), reverse);
}

// Packed sequences: which one starts, and which ends, at token i of tile p (-1: none).
// Returns, in every lane, whether there is any among the warp's.
__device__ __forceinline__ bool sequence_marks(const GlrArgs& a, int p, int i, int* starts, int* ends) {
    const int t = p * kTile + i;
    int s = -1, e = -1;
    if (t < a.T) {
        const mix::Span sp = mix::span_of(a.cu, a.n_seqs, a.T, t);
        if (sp.first == t) s = sp.n;
        if (sp.end == t + 1) e = sp.n;
    }
    starts[i] = s;
    ends[i] = e;
    return __any_sync(~0u, s >= 0 || e >= 0);
}

}  // namespace glr
}  // namespace gdn
