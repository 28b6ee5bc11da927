// C ABI of linear attention with a decay for each head (declared in include/gdn.h): argument checks, workspaces, dispatch.

#include "lin.h"

#include "internal.h"
#include "mixer_check.h"

namespace {

using gdn::LinTok;
using gdn::LinWalk;

struct Sizes {
    int B, T, Hk, H, dk, dv;
    const int32_t* cu;
    int n_seqs;
    int N() const { return cu ? n_seqs : B; }
    int64_t rows() const { return (int64_t)B * T; }
    int group() const { return H / Hk; }
};

gdn_status check_sizes(const char* fn, const Sizes& z, gdn_dtype dtype, gdn_algo algo) {
    if (!dtype_ok(dtype)) return fail(GDN_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
    if (algo != GDN_ALGO_AUTO && algo != GDN_ALGO_GENERIC && algo != GDN_ALGO_TCGEN05)
        return fail(GDN_ERR_INVALID_ARG, "%s: algo must be GDN_ALGO_AUTO, _GENERIC or _TCGEN05 (got %d)", fn, (int)algo);
    if (z.B < 1 || z.T < 0 || z.Hk < 1 || z.H < 1 || z.dk < 1 || z.dv < 1)
        return fail(GDN_ERR_INVALID_ARG, "%s: need B, H_k, H, d_k, d_v >= 1 and T >= 0 (got %d, %d, %d, %d, %d, %d)", fn, z.B,
                    z.Hk, z.H, z.dk, z.dv, z.T);
    if (z.H % z.Hk)
        return fail(GDN_ERR_INVALID_ARG, "%s: H=%d value heads are no multiple of H_k=%d key heads", fn, z.H, z.Hk);
    if (z.dk > 256 || z.dv > 256)
        return fail(GDN_ERR_UNSUPPORTED, "%s: head sizes must be 1..256 (got d_k=%d, d_v=%d)", fn, z.dk, z.dv);
    if (z.rows() > kMaxRows)
        return fail(GDN_ERR_UNSUPPORTED, "%s: B * T = %lld tokens is more than %lld", fn, (long long)z.rows(), (long long)kMaxRows);
    if (z.cu || z.n_seqs) {
        if (z.B != 1) return fail(GDN_ERR_INVALID_ARG, "%s: cu_seqlens needs B == 1 (got B=%d)", fn, z.B);
        if (z.n_seqs < 1) return fail(GDN_ERR_INVALID_ARG, "%s: cu_seqlens needs n_seqs >= 1 (got %d)", fn, z.n_seqs);
        if (!aligned(z.cu, 4)) return fail(GDN_ERR_INVALID_ARG, "%s: cu_seqlens is not 4-byte aligned", fn);
    }
    const int64_t most = (int64_t(1) << 31) - 1;       // blocks of a launch
    if ((int64_t)z.N() > most / (8 * (int64_t)z.H) || gdn::lin_slots(z.rows(), z.N(), gdn::kLinChunk) > most / z.H)
        return fail(GDN_ERR_UNSUPPORTED, "%s: %d sequences of %d heads need more than 2^31 blocks", fn, z.N(), z.H);
    if (z.rows() * z.H > (int64_t(1) << 40) / 256)
        return fail(GDN_ERR_UNSUPPORTED, "%s: tokens times heads is more than 2^32", fn);
    return GDN_OK;
}

gdn_status check_strides(const char* fn, const char* name, const LinTok& t, int d) {
    if (t.tok < d || t.head < d || t.tok > (int64_t(1) << 31) || t.head > (int64_t(1) << 31))
        return fail(GDN_ERR_INVALID_ARG, "%s: the token and head strides of %s must be %d..2^31 elements (got %lld, %lld)", fn,
                    name, d, (long long)t.tok, (long long)t.head);
    return GDN_OK;
}

LinWalk walk(const Sizes& z, const LinTok& a, const LinTok& b, const LinTok& c, int da, int dc, const float* g, int g_per_head,
             gdn_dtype dtype) {
    LinWalk w{};
    w.a = a; w.b = b; w.c = c; w.da = da; w.dc = dc;
    w.g = g;
    w.g_tok = g_per_head ? 0 : z.H;
    w.g_head = 1;
    w.cu = z.cu; w.n_seqs = z.n_seqs; w.B = z.B; w.T = z.T; w.H = z.H;
    w.bf16 = dtype == GDN_BF16;
    return w;
}
void state(LinWalk& w, const float* in, float* out, int rows_step, int cols_step) {
    w.s_in = in; w.s_out = out; w.s_r = rows_step; w.s_c = cols_step;
}

// The tensor cores, where the request fits them and sequences have at least 16 tokens on average.  They are the faster ones at any
// length, but round the scores to bf16, and a score among few has nothing beside it that its rounding would average out with (the
// queries' gradient of one token and four heads that share it was off by 5e-3 of its size); the generic walk rounds none, and is
// near for so few (forward, 16 heads of 128: one token 11.5 against 9.0 us; 16 tokens 13.2 against 9.1, 128 tokens 41.7 against
// 8.2; 256 sequences of 8 tokens 854 against 478).
gdn_status choose(const char* fn, gdn_algo algo, const Sizes& z, bool fits, bool& tensor) {
    if (algo == GDN_ALGO_TCGEN05 && !fits)
        return fail(GDN_ERR_UNSUPPORTED, "%s: the tensor-core path takes bf16, d_k up to 128, d_v up to 256 (128 backward) in steps of 8, and "
                    "rows, heads and outputs on 16-byte boundaries", fn);
    tensor = fits && algo != GDN_ALGO_GENERIC && (algo == GDN_ALGO_TCGEN05 || z.rows() >= 16 * (int64_t)z.N());
    return GDN_OK;
}

// Segments of the walks, one set of states for all walks of a call (they come one after another) and for either kind of walk.
struct Segments {
    int fwd[2], bwd[2];                                    // chunks of a segment (generic, tensor cores): columns of d_v, and d_k
    size_t states, kept, bytes;
    Segments(const Sizes& z, bool backward) {
        states = kept = 0;
        for (int tensor = 0; tensor < 2; ++tensor)
            for (int i = 0; i < 2; ++i) {
                const int da = i ? z.dv : z.dk, dc = i ? z.dk : z.dv;
                const int chunks = i && !backward ? 0 : gdn::lin_segment_chunks(z.rows(), z.N(), z.cu != nullptr, z.H, da, dc, tensor);
                (i ? bwd : fwd)[tensor] = chunks;
                if (chunks == 0) continue;
                const size_t slots = (size_t)gdn::lin_slots(z.rows(), z.N(), (int64_t)chunks * gdn::kLinChunk) * z.H;
                const size_t n = 4 * slots * gdn::lin_span_floats(da, dc, tensor), m = 4 * slots;
                states = n > states ? n : states;
                kept = m > kept ? m : kept;
            }
        states = (states + 255) / 256 * 256;
        kept = (kept + 255) / 256 * 256;
        bytes = states + kept;
    }
    void put(LinWalk& w, void* base, bool tensor, const int (&chunks)[2]) const {
        if (chunks[tensor] == 0) return;
        w.seg_chunks = chunks[tensor];
        w.seg_states = static_cast<float*>(base);
        w.seg_kept = reinterpret_cast<float*>(static_cast<char*>(base) + states);
    }
};

// Parts of the backward's workspace, each a multiple of 256 bytes (for either walk: which one it is goes by the buffers too).
struct BwdParts {
    size_t plus, minus, pairs, spans, anchors, part, group, bytes;
    Segments segments;
    explicit BwdParts(const Sizes& z) : segments(z, true) {
        size_t at = segments.bytes;
        auto take = [&](size_t n) {
            const size_t here = at;
            at += (n + 255) / 256 * 256;
            return here;
        };
        const size_t slots = (size_t)gdn::lin_span_slots(z.rows(), z.N()), heads = (size_t)z.H;
        const size_t blocks = (size_t)gdn::lin_blocks(z.dk, false);
        const size_t span = gdn::lin_span_floats(z.dv, z.dk, false), tc = gdn::lin_span_floats(z.dv, z.dk, true);
        plus = take(4 * blocks * heads * (size_t)z.rows());
        minus = take(4 * blocks * heads * (size_t)z.rows());
        pairs = take(4 * 2 * blocks * heads * (size_t)z.rows());     // (the tensor cores' are one array, the generic walks' two a block)
        spans = take(4 * slots * heads * (span > tc ? span : tc));
        const size_t tc_blocks = 8 * (size_t)gdn::lin_blocks(z.dk, true);
        anchors = take(4 * slots * heads * (blocks > tc_blocks ? blocks : tc_blocks));
        part = take(4 * slots * heads);
        group = take(z.group() > 1 ? 4 * (size_t)z.rows() * heads * (size_t)z.dk : 0);
        bytes = at;
    }
};

}  // namespace

extern "C" {

gdn_status lin_workspace_size(int backward, int B, int T, int H_k, int H, int d_k, int d_v, int n_seqs, size_t* bytes) {
    const char* fn = "lin_workspace_size";
    if (!bytes) return fail(GDN_ERR_INVALID_ARG, "%s: bytes is NULL", fn);
    if (n_seqs < 0) return fail(GDN_ERR_INVALID_ARG, "%s: n_seqs must be >= 0 (got %d)", fn, n_seqs);
    const Sizes z{B, T, H_k, H, d_k, d_v, n_seqs > 0 ? reinterpret_cast<const int32_t*>(uintptr_t(1) << 20) : nullptr, n_seqs};
    GDN_TRY(check_sizes(fn, z, GDN_F32, GDN_ALGO_AUTO));
    *bytes = backward ? BwdParts(z).bytes : Segments(z, false).bytes;
    return ok();
}

gdn_status lin_chunk_fwd(const void* q, const void* k, const void* v, const float* g, int g_per_head, float scale,
                         const float* initial_state, float* final_state, const int32_t* cu_seqlens, int n_seqs, void* o,
                         int B, int T, int H_k, int H, int d_k, int d_v, int64_t q_token_stride, int64_t q_head_stride,
                         int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                         gdn_dtype dtype, gdn_algo algo, void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "lin_chunk_fwd";
    const Sizes z{B, T, H_k, H, d_k, d_v, cu_seqlens, cu_seqlens ? n_seqs : 0};
    GDN_TRY(check_sizes(fn, z, dtype, algo));
    const size_t es = size_of(dtype);
    const LinTok tq{q, q_token_stride, q_head_stride, z.group()}, tk{k, k_token_stride, k_head_stride, z.group()};
    const LinTok tv{v, v_token_stride, v_head_stride, 1};
    GDN_TRY(check_strides(fn, "q", tq, d_k));
    GDN_TRY(check_strides(fn, "k", tk, d_k));
    GDN_TRY(check_strides(fn, "v", tv, d_v));
    if (T > 0) {
        GDN_TRY(need(fn, "q", q, es));
        GDN_TRY(need(fn, "k", k, es));
        GDN_TRY(need(fn, "v", v, es));
        GDN_TRY(need(fn, "g", g, 4));
        GDN_TRY(need(fn, "o", o, es));
    }
    GDN_TRY(may(fn, "initial_state", initial_state, 4));
    GDN_TRY(may(fn, "final_state", final_state, 4));
    LinWalk w = walk(z, tq, tk, tv, d_k, d_v, g, g_per_head, dtype);
    w.s_intra = w.s_inter = scale;
    w.s_state = 1.f;
    state(w, initial_state, final_state, d_v, 1);
    w.out = o;
    w.out_f32 = dtype == GDN_F32;
    bool tensor = false;
    GDN_TRY(choose(fn, algo, z, gdn::lin_tensor_fits(w), tensor));
    Workspace ws;
    const Segments segments(z, false);
    GDN_TRY(ws.get(fn, workspace, workspace_bytes, segments.fwd[tensor] ? segments.bytes : 0, static_cast<cudaStream_t>(stream)));
    segments.put(w, ws.ptr, tensor, segments.fwd);
    w.test_stall = tensor && gdn::take_test_injection(GDN_TEST_LIN_STALL);
    return finish(fn, tensor ? gdn::launch_lin_walk_tensor(w, false, ws.s) : gdn::launch_lin_walk_generic(w, false, ws.s), ws);
}

gdn_status lin_chunk_bwd(const void* q, const void* k, const void* v, const float* g, int g_per_head, float scale,
                         const float* initial_state, const void* grad_o, const float* grad_final_state,
                         const int32_t* cu_seqlens, int n_seqs, void* grad_q, void* grad_k, void* grad_v, float* grad_g,
                         float* grad_initial_state, int B, int T, int H_k, int H, int d_k, int d_v, int64_t q_token_stride,
                         int64_t q_head_stride, int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                         int64_t v_head_stride, gdn_dtype dtype, gdn_algo algo, void* workspace, size_t workspace_bytes,
                         void* stream) {
    const char* fn = "lin_chunk_bwd";
    const Sizes z{B, T, H_k, H, d_k, d_v, cu_seqlens, cu_seqlens ? n_seqs : 0};
    GDN_TRY(check_sizes(fn, z, dtype, algo));
    const size_t es = size_of(dtype);
    const int group = z.group();
    const LinTok tq{q, q_token_stride, q_head_stride, group}, tk{k, k_token_stride, k_head_stride, group};
    const LinTok tv{v, v_token_stride, v_head_stride, 1}, to{grad_o, (int64_t)H * d_v, d_v, 1};
    GDN_TRY(check_strides(fn, "q", tq, d_k));
    GDN_TRY(check_strides(fn, "k", tk, d_k));
    GDN_TRY(check_strides(fn, "v", tv, d_v));
    if (T > 0) {
        GDN_TRY(need(fn, "q", q, es));
        GDN_TRY(need(fn, "k", k, es));
        GDN_TRY(need(fn, "v", v, es));
        GDN_TRY(need(fn, "g", g, 4));
        GDN_TRY(need(fn, "grad_o", grad_o, es));
        GDN_TRY(need(fn, "grad_q", grad_q, es));
        GDN_TRY(need(fn, "grad_k", grad_k, es));
        GDN_TRY(need(fn, "grad_v", grad_v, es));
    }
    if (T > 0 || g_per_head) GDN_TRY(need(fn, "grad_g", grad_g, 4));
    GDN_TRY(may(fn, "initial_state", initial_state, 4));
    GDN_TRY(may(fn, "grad_final_state", grad_final_state, 4));
    GDN_TRY(may(fn, "grad_initial_state", grad_initial_state, 4));
    const BwdParts parts(z);
    Workspace ws;
    GDN_TRY(ws.get(fn, workspace, workspace_bytes, parts.bytes, static_cast<cudaStream_t>(stream)));
    char* base = static_cast<char*>(ws.ptr);
    auto part = [&](size_t at) { return reinterpret_cast<float*>(base + at); };

    float* pairs = part(parts.pairs);
    float* pairs_minus = pairs + (int64_t)gdn::lin_blocks(d_k, false) * H * z.rows();
    // dq, with the states at the spans' starts on the way
    LinWalk wq = walk(z, to, tv, tk, d_v, d_k, g, g_per_head, dtype);
    wq.s_intra = wq.s_inter = scale;
    wq.s_state = 1.f;
    state(wq, initial_state, nullptr, 1, d_v);
    wq.out = group > 1 ? part(parts.group) : grad_q;
    wq.out_f32 = group > 1 || dtype == GDN_F32;
    wq.x = tq;
    wq.dots = part(parts.plus);
    wq.pair_dots = pairs;
    wq.spans = part(parts.spans);
    // dk, from the last token to the first, with the states' inner products
    LinWalk wk = walk(z, tv, to, tq, d_v, d_k, g, g_per_head, dtype);
    wk.rev = 1;
    wk.s_intra = wk.s_state = scale;
    wk.s_inter = 1.f;
    state(wk, grad_final_state, nullptr, 1, d_v);
    wk.out = group > 1 ? part(parts.group) : grad_k;
    wk.out_f32 = group > 1 || dtype == GDN_F32;
    wk.x = tk;
    wk.dots = part(parts.minus);
    wk.pair_dots = pairs_minus;
    wk.spans = part(parts.spans);
    wk.anchors = part(parts.anchors);
    // dv, and the gradient of the initial state
    LinWalk wv = walk(z, tk, tq, to, d_k, d_v, g, g_per_head, dtype);
    wv.rev = 1;
    wv.s_intra = wv.s_state = scale;
    wv.s_inter = 1.f;
    state(wv, grad_final_state, grad_initial_state, d_v, 1);
    wv.out = grad_v;
    wv.out_f32 = dtype == GDN_F32;
    bool tensor = false;
    if (T > 0)
        GDN_TRY(choose(fn, algo, z, gdn::lin_tensor_fits(wq) && gdn::lin_tensor_fits(wk) && gdn::lin_tensor_fits(wv) &&
                       aligned(grad_q, 16) && aligned(grad_k, 16), tensor));
    wq.fine = wk.fine = g_per_head != 0;
    parts.segments.put(wq, base, tensor, parts.segments.bwd);
    parts.segments.put(wk, base, tensor, parts.segments.bwd);
    parts.segments.put(wv, base, tensor, parts.segments.fwd);
    auto run = [&](const LinWalk& w, bool behind) {
        return tensor ? gdn::launch_lin_walk_tensor(w, behind, ws.s) : gdn::launch_lin_walk_generic(w, behind, ws.s);
    };
    cudaError_t e = run(wq, false);
    if (e == cudaSuccess && group > 1)
        e = gdn::launch_lin_group_sum(part(parts.group), grad_q, wq.bf16, z.rows(), H_k, group, d_k, ws.s);
    if (e == cudaSuccess) e = run(wk, group == 1);         // (else in the place that the sum over the group still reads)
    if (e == cudaSuccess && group > 1)
        e = gdn::launch_lin_group_sum(part(parts.group), grad_k, wk.bf16, z.rows(), H_k, group, d_k, ws.s);
    if (e == cudaSuccess) e = run(wv, true);
    if (tensor && e == cudaSuccess)
        e = gdn::launch_lin_pairs({tq, tk, tv, to, d_k, d_v, scale, g, wq.g_tok, wq.g_head, z.cu, z.n_seqs, B, T, H, pairs}, ws.s);
    gdn::LinDg d{};
    d.plus = part(parts.plus);
    d.minus = part(parts.minus);
    d.pairs = pairs;
    d.pairs_minus = tensor ? nullptr : pairs_minus;
    d.anchors = part(parts.anchors);
    d.blocks = gdn::lin_blocks(d_k, tensor);
    d.pair_blocks = tensor ? 1 : d.blocks;
    d.chunk = tensor ? gdn::kLinChunk : gdn::kLinGenericChunk;
    d.anchor_blocks = tensor ? 8 * d.blocks : d.blocks;
    d.dg = grad_g;
    d.per_head = g_per_head != 0;
    d.part = part(parts.part);
    d.cu = z.cu;
    d.n_seqs = z.n_seqs;
    d.B = B;
    d.T = T;
    d.H = H;
    if (e == cudaSuccess) e = gdn::launch_lin_dg(d, ws.s);
    return finish(fn, e, ws);
}

gdn_status lin_recurrent_step(const void* q, const void* k, const void* v, const float* g, int g_per_head, float scale,
                              const float* state, float* state_out, void* o, int N, int H_k, int H, int d_k, int d_v,
                              int64_t q_token_stride, int64_t q_head_stride, int64_t k_token_stride, int64_t k_head_stride,
                              int64_t v_token_stride, int64_t v_head_stride, gdn_dtype dtype, void* stream) {
    const char* fn = "lin_recurrent_step";
    const Sizes z{N, 1, H_k, H, d_k, d_v, nullptr, 0};
    GDN_TRY(check_sizes(fn, z, dtype, GDN_ALGO_AUTO));
    const size_t es = size_of(dtype);
    const LinTok tq{q, q_token_stride, q_head_stride, z.group()}, tk{k, k_token_stride, k_head_stride, z.group()};
    const LinTok tv{v, v_token_stride, v_head_stride, 1};
    GDN_TRY(check_strides(fn, "q", tq, d_k));
    GDN_TRY(check_strides(fn, "k", tk, d_k));
    GDN_TRY(check_strides(fn, "v", tv, d_v));
    GDN_TRY(need(fn, "q", q, es));
    GDN_TRY(need(fn, "k", k, es));
    GDN_TRY(need(fn, "v", v, es));
    GDN_TRY(need(fn, "g", g, 4));
    GDN_TRY(need(fn, "state", state, 4));
    GDN_TRY(need(fn, "state_out", state_out, 4));
    GDN_TRY(need(fn, "o", o, es));
    gdn::LinStepArgs a{tq, tk, tv, g, g_per_head ? 0 : (int64_t)H, 1, scale, state, state_out, o, N, H, d_k, d_v, dtype == GDN_BF16};
    const cudaError_t e = gdn::launch_lin_step(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}

}  // extern "C"
