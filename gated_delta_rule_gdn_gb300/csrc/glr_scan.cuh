// Shared parts of the gated linear recurrence's scans (glr_scan.cu, glr_scan_bwd.cu): the tiling, and the carry of a
// tile from the tiles before it.
//
// A row of T tokens is cut into tiles of 64 tokens x 32 V channels, a block each; a warp takes 8 consecutive tokens of
// the tile, a lane V channels, and holds them in registers.  The recurrence over a run of tokens is the map
// h -> A h + H; a run in which a sequence starts (backward: ends) forgets h altogether, which is written A = -1 (decays
// are never negative), so that a state that is not a number stays in its own sequence.
//
// The carry into tile p (in scan order) is, in a fixed association whatever the timing, so that results do not change
// from run to run:
//   the state at the start of its group of kGroup tiles, then the maps of the group's tiles before it, composed first.
// A tile publishes its map as soon as it has it; the last of a group publishes the next group's starting state.  So the
// serial chain of a row is T / (64 kGroup) hops, and each byte of the inputs is read once.  Tiles take tickets in scan
// order, so every tile that a block waits for has been started before it; waits are bounded all the same.
#pragma once

#include "glr_math.cuh"
#include "mixer.h"
#include "mixer_common.cuh"

namespace gdn {
namespace glr {

constexpr int kWarps = 8, kRun = 8;              // a warp's run of tokens
constexpr int kTile = kWarps * kRun;
static_assert(kTile == kGlrTile, "checkpoints are tile entries");
constexpr int kGroup = 16;
constexpr unsigned long long kWaitNs = 2000000000ull;

// Workspace of one scan: [ticket, gave-up flag, map flags [chains][tiles], state flags [chains][groups]] zeroed before
// the launch, then the maps and the states.
struct Exchange {
    unsigned* ticket;
    unsigned* gave_up;
    unsigned* map_flag;
    unsigned* state_flag;
    float2* map;            // [tiles][chains][width]
    float* state;           // [groups][chains][width]
    int tiles, groups, chains;
};

struct Layout {
    size_t flag_bytes, map_off, state_off, bytes;
    int tiles, groups, chains;
};
inline Layout layout(int B, int T, int D, int width) {
    Layout l;
    l.tiles = T > kTile ? (T + kTile - 1) / kTile : 1;
    l.groups = (l.tiles + kGroup - 1) / kGroup;
    l.chains = B * ((D + width - 1) / width);
    if (l.tiles == 1) {                          // nothing to exchange
        l.flag_bytes = l.map_off = l.state_off = l.bytes = 0;
        return l;
    }
    const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    l.flag_bytes = up((2 + (size_t)l.chains * (l.tiles + l.groups)) * sizeof(unsigned));
    l.map_off = l.flag_bytes;
    l.state_off = up(l.map_off + (size_t)l.tiles * l.chains * width * sizeof(float2));
    l.bytes = up(l.state_off + (size_t)l.groups * l.chains * width * sizeof(float));
    return l;
}
inline Exchange exchange(const Layout& l, void* ws) {
    Exchange x{};
    char* p = static_cast<char*>(ws);
    x.tiles = l.tiles; x.groups = l.groups; x.chains = l.chains;
    if (l.tiles == 1) return x;
    x.ticket = reinterpret_cast<unsigned*>(p);
    x.gave_up = x.ticket + 1;
    x.map_flag = x.ticket + 2;
    x.state_flag = x.map_flag + (size_t)l.chains * l.tiles;
    x.map = reinterpret_cast<float2*>(p + l.map_off);
    x.state = reinterpret_cast<float*>(p + l.state_off);
    return x;
}

__device__ __forceinline__ float apply(float A, float H, float h) { return A < 0.f ? H : fmaf(A, h, H); }
__device__ __forceinline__ float both(float A1, float A2) { return A1 < 0.f || A2 < 0.f ? -1.f : A1 * A2; }

__device__ __forceinline__ unsigned load_acquire(const unsigned* p) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void store_release(unsigned* p, unsigned v) {
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
// Wait until *p is set.  Gives up after kWaitNs, or soon after another block has; the call's outputs are then
// unspecified and *status says so.
__device__ __forceinline__ void wait_flag(const unsigned* p, unsigned* gave_up, unsigned* status) {
    if (load_acquire(p)) return;
    unsigned long long t0, t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
    while (true) {
        for (int i = 0; i < 64; ++i)
            if (load_acquire(p)) return;
        asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
        if (t - t0 > kWaitNs || load_acquire(gave_up)) {
            atomicExch(gave_up, 1u);
            atomicOr(status, 1u);
            return;
        }
    }
}

// The carry into tile p of a chain.  Called by the whole block; threads below `width` pass their channel's map (A, H)
// of the tile and the state `first` before tile 0 of the row, and get the carry.
__device__ __forceinline__ float carry_in(const Exchange& x, int width, int p, int chain, float A, float H, float first,
                                          bool publish, unsigned* status) {
    const int tid = threadIdx.x, start = p / kGroup * kGroup, group = p / kGroup;
    const bool more = p + 1 < x.tiles, closes = more && p + 1 == start + kGroup;
    const size_t at = (size_t)chain * width + tid, row = (size_t)x.chains * width;
    if (more && !closes) {
        if (tid < width) __stcg(&x.map[p * row + at], make_float2(A, H));
        __syncthreads();
        if (tid == 0 && publish) {
            __threadfence();
            store_release(&x.map_flag[(size_t)chain * x.tiles + p], 1u);
        }
    }
    float cA = 1.f, cH = 0.f;
    if (p > start) {
        if (tid < p - start) wait_flag(&x.map_flag[(size_t)chain * x.tiles + start + tid], x.gave_up, status);
        __syncthreads();
        if (tid < width) {
            float2 m[kGroup - 1];
#pragma unroll
            for (int j = 0; j < kGroup - 1; ++j)
                m[j] = start + j < p ? __ldcg(&x.map[(start + j) * row + at]) : make_float2(1.f, 0.f);
#pragma unroll
            for (int j = 0; j < kGroup - 1; ++j) {
                cH = apply(m[j].x, m[j].y, cH);
                cA = both(cA, m[j].x);
            }
        }
    }
    if (group > 0) {
        if (tid == 0) wait_flag(&x.state_flag[(size_t)chain * x.groups + group], x.gave_up, status);
        __syncthreads();
        if (tid < width) first = __ldcg(&x.state[group * row + at]);
    }
    const float carry = apply(cA, cH, first);
    if (closes) {
        if (tid < width) __stcg(&x.state[(group + 1) * row + at], apply(A, H, carry));
        __syncthreads();
        if (tid == 0 && publish) {
            __threadfence();
            store_release(&x.state_flag[(size_t)chain * x.groups + group + 1], 1u);
        }
    }
    return carry;
}

struct Channel { float neg_eA, dt; };   // -exp(A_log) (0: g is log a) and dt_bias of a channel
__device__ __forceinline__ Channel channel(const float* A_log, const float* dt_bias, int c) {
    return {A_log ? -expf(A_log[c]) : 0.f, dt_bias ? dt_bias[c] : 0.f};
}

}  // namespace glr
}  // namespace gdn
