// C ABI of the operators around the delta rule (declared in include/gdn.h): argument checks and dispatch of the gated
// linear recurrence, the query/key head norm with rotation, and the short convolution.

#include <cuda_runtime.h>

#include <cmath>

#include "../../include/gdn.h"
#include "api_util.h"
#include "internal.h"
#include "mixer.h"
#include "mixer_check.h"

namespace {

using gdn::aligned;
using gdn::cuda_fail;
using gdn::dtype_ok;
using gdn::fail;
using gdn::ok;

gdn_status check_sizes(const char* fn, int B, int T, int D, const int32_t* cu, int n_seqs) {
    if (B < 1 || T < 0 || D < 1)
        return fail(GDN_ERR_INVALID_ARG, "%s: need B >= 1, T >= 0, D >= 1 (got B=%d T=%d D=%d)", fn, B, T, D);
    if ((int64_t)B * T > kMaxRows)
        return fail(GDN_ERR_UNSUPPORTED, "%s: B * T = %lld tokens is more than %lld", fn, (long long)B * T,
                    (long long)kMaxRows);
    if ((int64_t)B * (T > 0 ? T : 1) > (int64_t(1) << 37) / D || (cu && (int64_t)n_seqs > (int64_t(1) << 37) / D))
        return fail(GDN_ERR_UNSUPPORTED, "%s: a tensor has more than 2^37 elements", fn);
    if ((int64_t)B * (T / 64 + 1) > ((int64_t(1) << 31) - 1) / (D / 32 + 1))     // one block per 64 tokens x 32 channels
        return fail(GDN_ERR_UNSUPPORTED, "%s: B=%d T=%d D=%d needs more than 2^31 blocks", fn, B, T, D);
    if (cu) {
        if (B != 1) return fail(GDN_ERR_INVALID_ARG, "%s: cu_seqlens needs B == 1 (got B=%d)", fn, B);
        if (n_seqs < 1) return fail(GDN_ERR_INVALID_ARG, "%s: cu_seqlens needs n_seqs >= 1 (got %d)", fn, n_seqs);
        if (!aligned(cu, 4)) return fail(GDN_ERR_INVALID_ARG, "%s: cu_seqlens is not 4-byte aligned", fn);
    }
    return GDN_OK;
}

gdn_status check_ld(const char* fn, const char* name, int64_t ld, int64_t least) {
    if (ld < least || ld > (int64_t(1) << 31))
        return fail(GDN_ERR_INVALID_ARG, "%s: the row stride of %s must be %lld..2^31 elements (got %lld)", fn, name,
                    (long long)least, (long long)ld);
    return GDN_OK;
}

// The types, gate parameters and row strides shared by the recurrence's entry points.
gdn_status check_glr(const char* fn, const float* A_log, const float* dt_bias, const void* gi, int D, int64_t ld_x,
                     int64_t ld_g, int64_t ld_i, gdn_dtype dtype, gdn_dtype g_dtype) {
    if (!dtype_ok(dtype)) return fail(GDN_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
    if (!dtype_ok(g_dtype)) return fail(GDN_ERR_INVALID_ARG, "%s: unknown g_dtype %d", fn, (int)g_dtype);
    if (dtype == GDN_F32 && g_dtype == GDN_BF16)
        return fail(GDN_ERR_UNSUPPORTED, "%s: bf16 gates go with bf16 inputs (x is fp32)", fn);
    if (dt_bias && !A_log) return fail(GDN_ERR_INVALID_ARG, "%s: dt_bias is given without A_log", fn);
    GDN_TRY(may(fn, "A_log", A_log, 4));
    GDN_TRY(may(fn, "dt_bias", dt_bias, 4));
    GDN_TRY(check_ld(fn, "x", ld_x, D));
    GDN_TRY(check_ld(fn, "g", ld_g, D));
    if (gi) GDN_TRY(check_ld(fn, "in_gate", ld_i, D));
    return GDN_OK;
}

gdn_status check_conv(const char* fn, int activation, int W, int D, int64_t ld_x, gdn_dtype dtype) {
    if (!dtype_ok(dtype)) return fail(GDN_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
    if (activation != GDN_ACT_NONE && activation != GDN_ACT_SILU)
        return fail(GDN_ERR_INVALID_ARG, "%s: unknown activation %d", fn, activation);
    if (W < 2 || W > 4) return fail(GDN_ERR_UNSUPPORTED, "%s: the width must be 2, 3 or 4 (got %d)", fn, W);
    return check_ld(fn, "x", ld_x, D);
}

gdn_status check_qk(const char* fn, gdn::QkNormArgs& a, int norm, int T, int d, gdn_dtype dtype) {
    if (!dtype_ok(dtype)) return fail(GDN_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
    if (norm != GDN_NORM_RMS && norm != GDN_NORM_L2) return fail(GDN_ERR_INVALID_ARG, "%s: unknown norm %d", fn, norm);
    if (a.n < 0 || a.H[0] < 1 || a.H[1] < 1 || T < 1)
        return fail(GDN_ERR_INVALID_ARG, "%s: need n_tokens >= 0, T >= 1 and at least one query and one key head (got "
                    "%lld, %d, %d, %d)", fn, (long long)a.n, T, a.H[0], a.H[1]);
    if (d < 1 || d > 256) return fail(GDN_ERR_UNSUPPORTED, "%s: the head size must be 1..256 (got %d)", fn, d);
    if (a.n > kMaxRows / ((int64_t)a.H[0] + a.H[1]))
        return fail(GDN_ERR_UNSUPPORTED, "%s: tokens times heads is more than %lld", fn, (long long)kMaxRows);
    if (!(a.eps > 0.f) || !std::isfinite(a.eps))
        return fail(GDN_ERR_INVALID_ARG, "%s: eps must be positive and finite", fn);
    if (a.rot < 0 || a.rot > d || a.rot % 2)
        return fail(GDN_ERR_INVALID_ARG, "%s: rotary_dim must be even and 0..d (got %d, d=%d)", fn, a.rot, d);
    if (a.rot > 0) {
        GDN_TRY(need(fn, "cos", a.cos, 4));
        GDN_TRY(need(fn, "sin", a.sin, 4));
        if (a.n_pos < 1) return fail(GDN_ERR_INVALID_ARG, "%s: the rotation table needs n_pos >= 1 (got %d)", fn, a.n_pos);
        if (!a.pos && T > a.n_pos)
            return fail(GDN_ERR_INVALID_ARG, "%s: %d tokens do not fit the rotation table of %d positions", fn, T, a.n_pos);
    }
    GDN_TRY(may(fn, "positions", a.pos, 4));
    const size_t es = size_of(dtype);
    const char* names[2] = {"q", "k"};
    for (int i = 0; i < 2; ++i) {
        if (a.n > 0) GDN_TRY(need(fn, names[i], a.in[i], es));
        GDN_TRY(may(fn, i ? "k_weight" : "q_weight", a.w[i], 4));
        if (a.head_stride[i] < d || a.head_stride[i] > (int64_t(1) << 31) || a.tok_stride[i] > (int64_t(1) << 31) ||
            a.tok_stride[i] < d)
            return fail(GDN_ERR_INVALID_ARG, "%s: the token and head strides of %s must be d..2^31 elements", fn, names[i]);
    }
    a.c = norm == GDN_NORM_RMS ? 1.f / (float)d : 1.f;
    a.T = T;
    a.d = d;
    a.bf16 = dtype == GDN_BF16;
    return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status glr_workspace_size(int backward, int B, int T, int D, int n_seqs, size_t* bytes) {
    const char* fn = "glr_workspace_size";
    if (!bytes) return fail(GDN_ERR_INVALID_ARG, "%s: bytes is NULL", fn);
    if (n_seqs < 0) return fail(GDN_ERR_INVALID_ARG, "%s: n_seqs must be >= 0 (got %d)", fn, n_seqs);
    gdn::GlrArgs a{};
    a.B = B; a.T = T; a.D = D; a.n_seqs = n_seqs;
    a.cu = n_seqs > 0 ? reinterpret_cast<const int32_t*>(uintptr_t(1) << 20) : nullptr;
    GDN_TRY(check_sizes(fn, B, T, D, a.cu, n_seqs));
    *bytes = gdn::glr_workspace_bytes(a, backward != 0);
    return ok();
}

gdn_status glr_scan_fwd(const void* x, const void* g, const void* in_gate, const float* A_log, const float* dt_bias,
                        int normalize, const float* initial_state, float* final_state, const int32_t* cu_seqlens,
                        int n_seqs, void* o, float* checkpoints, int B, int T, int D, int64_t ld_x, int64_t ld_g,
                        int64_t ld_i, gdn_dtype dtype, gdn_dtype g_dtype, void* workspace, size_t workspace_bytes,
                        void* stream) {
    const char* fn = "glr_scan_fwd";
    GDN_TRY(check_sizes(fn, B, T, D, cu_seqlens, n_seqs));
    GDN_TRY(check_glr(fn, A_log, dt_bias, in_gate, D, ld_x, ld_g, ld_i, dtype, g_dtype));
    const size_t es = size_of(dtype), gs = size_of(g_dtype);
    if (T > 0) {
        GDN_TRY(need(fn, "x", x, es));
        GDN_TRY(need(fn, "g", g, gs));
        GDN_TRY(need(fn, "o", o, es));
    }
    GDN_TRY(may(fn, "in_gate", in_gate, es));
    GDN_TRY(may(fn, "initial_state", initial_state, 4));
    GDN_TRY(may(fn, "final_state", final_state, 4));
    GDN_TRY(may(fn, "checkpoints", checkpoints, 4));
    gdn::GlrArgs a{};
    a.x = x; a.g = g; a.gi = in_gate; a.A_log = A_log; a.dt_bias = dt_bias; a.normalize = normalize != 0;
    a.h0 = initial_state; a.hT = final_state; a.cu = cu_seqlens; a.n_seqs = n_seqs; a.o = o; a.ckpt = checkpoints;
    a.B = B; a.T = T; a.D = D; a.ldx = ld_x; a.ldg = ld_g; a.ldi = ld_i;
    a.bf16 = dtype == GDN_BF16; a.g_bf16 = g_dtype == GDN_BF16;
    Workspace ws;
    GDN_TRY(ws.get(fn, workspace, workspace_bytes, gdn::glr_workspace_bytes(a, false), static_cast<cudaStream_t>(stream)));
    a.ws = ws.ptr;
    a.test_stall = gdn::take_test_injection(GDN_TEST_GLR_STALL);
    return finish(fn, gdn::launch_glr_fwd(a, ws.s), ws);
}

gdn_status glr_scan_bwd(const void* x, const void* g, const void* in_gate, const float* A_log, const float* dt_bias,
                        int normalize, const float* initial_state, const void* grad_o, const float* grad_final_state,
                        const int32_t* cu_seqlens, int n_seqs, const float* checkpoints, void* grad_x, void* grad_g,
                        void* grad_in_gate, float* grad_initial_state, float* grad_A_log, float* grad_dt_bias, int B,
                        int T, int D, int64_t ld_x, int64_t ld_g, int64_t ld_i, gdn_dtype dtype, gdn_dtype g_dtype,
                        void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "glr_scan_bwd";
    GDN_TRY(check_sizes(fn, B, T, D, cu_seqlens, n_seqs));
    GDN_TRY(check_glr(fn, A_log, dt_bias, in_gate, D, ld_x, ld_g, ld_i, dtype, g_dtype));
    const size_t es = size_of(dtype), gs = size_of(g_dtype);
    if (T > 0) {
        GDN_TRY(need(fn, "x", x, es));
        GDN_TRY(need(fn, "g", g, gs));
        GDN_TRY(need(fn, "grad_o", grad_o, es));
        GDN_TRY(need(fn, "grad_x", grad_x, es));
        GDN_TRY(need(fn, "grad_g", grad_g, gs));
        if (in_gate) GDN_TRY(need(fn, "grad_in_gate", grad_in_gate, es));
    }
    GDN_TRY(may(fn, "in_gate", in_gate, es));
    if (A_log) GDN_TRY(need(fn, "grad_A_log", grad_A_log, 4));
    if (grad_dt_bias && !dt_bias) return fail(GDN_ERR_INVALID_ARG, "%s: grad_dt_bias needs dt_bias", fn);
    GDN_TRY(may(fn, "grad_dt_bias", grad_dt_bias, 4));
    GDN_TRY(may(fn, "initial_state", initial_state, 4));
    GDN_TRY(may(fn, "grad_final_state", grad_final_state, 4));
    GDN_TRY(may(fn, "grad_initial_state", grad_initial_state, 4));
    GDN_TRY(may(fn, "checkpoints", checkpoints, 4));
    gdn::GlrArgs a{};
    a.x = x; a.g = g; a.gi = in_gate; a.A_log = A_log; a.dt_bias = dt_bias; a.normalize = normalize != 0;
    a.h0 = initial_state; a.cu = cu_seqlens; a.n_seqs = n_seqs; a.ckpt = const_cast<float*>(checkpoints);
    a.dO = grad_o; a.dhT = grad_final_state; a.dx = grad_x; a.dg = grad_g; a.di = grad_in_gate;
    a.dh0 = grad_initial_state; a.dA = A_log ? grad_A_log : nullptr; a.ddt = grad_dt_bias;
    a.B = B; a.T = T; a.D = D; a.ldx = ld_x; a.ldg = ld_g; a.ldi = ld_i;
    a.bf16 = dtype == GDN_BF16; a.g_bf16 = g_dtype == GDN_BF16;
    Workspace ws;
    GDN_TRY(ws.get(fn, workspace, workspace_bytes, gdn::glr_workspace_bytes(a, true), static_cast<cudaStream_t>(stream)));
    a.ws = ws.ptr;
    return finish(fn, gdn::launch_glr_bwd(a, ws.s), ws);
}

gdn_status glr_step(const void* x, const void* g, const void* in_gate, const float* A_log, const float* dt_bias,
                    int normalize, const float* state, float* state_out, void* o, int N, int D, int64_t ld_x,
                    int64_t ld_g, int64_t ld_i, gdn_dtype dtype, gdn_dtype g_dtype, void* stream) {
    const char* fn = "glr_step";
    GDN_TRY(check_sizes(fn, N, 1, D, nullptr, 0));
    GDN_TRY(check_glr(fn, A_log, dt_bias, in_gate, D, ld_x, ld_g, ld_i, dtype, g_dtype));
    const size_t es = size_of(dtype);
    GDN_TRY(need(fn, "x", x, es));
    GDN_TRY(need(fn, "g", g, size_of(g_dtype)));
    GDN_TRY(may(fn, "in_gate", in_gate, es));
    GDN_TRY(need(fn, "state", state, 4));
    GDN_TRY(need(fn, "state_out", state_out, 4));
    GDN_TRY(need(fn, "o", o, es));
    gdn::GlrStepArgs a{x, g, in_gate, A_log, dt_bias, normalize != 0, state, state_out, o, N, D, ld_x, ld_g, ld_i,
                       dtype == GDN_BF16, g_dtype == GDN_BF16};
    const cudaError_t e = gdn::launch_glr_step(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}

gdn_status gdn_qk_norm_fwd(const void* q, const void* k, const float* q_weight, const float* k_weight, gdn_norm norm,
                           float eps, const float* cos, const float* sin, int n_pos, int rotary_dim, int interleaved,
                           const int32_t* positions, void* q_out, void* k_out, int64_t n_tokens, int T, int H_q,
                           int H_k, int d, int64_t q_token_stride, int64_t q_head_stride, int64_t k_token_stride,
                           int64_t k_head_stride, gdn_dtype dtype, void* stream) {
    const char* fn = "gdn_qk_norm_fwd";
    gdn::QkNormArgs a{{q, k}, {}, {q_out, k_out}, {q_weight, k_weight}, {}, {q_token_stride, k_token_stride},
                      {q_head_stride, k_head_stride}, {H_q, H_k}, n_tokens, 0, 0, 0.f, eps, cos, sin, n_pos,
                      rotary_dim, interleaved != 0, positions, 0, nullptr};
    GDN_TRY(check_qk(fn, a, norm, T, d, dtype));
    if (a.n == 0) return ok();
    GDN_TRY(need(fn, "q_out", q_out, size_of(dtype)));
    GDN_TRY(need(fn, "k_out", k_out, size_of(dtype)));
    const cudaError_t e = gdn::launch_qk_norm_fwd(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}

gdn_status gdn_qk_norm_workspace_size(int64_t n_tokens, int H_q, int H_k, int d, size_t* bytes) {
    const char* fn = "gdn_qk_norm_workspace_size";
    if (!bytes) return fail(GDN_ERR_INVALID_ARG, "%s: bytes is NULL", fn);
    gdn::QkNormArgs a{};
    a.n = n_tokens;
    a.H[0] = H_q;
    a.H[1] = H_k;
    a.eps = 1.f;
    for (int i = 0; i < 2; ++i) {
        a.in[i] = reinterpret_cast<const void*>(uintptr_t(1) << 20);
        a.tok_stride[i] = a.head_stride[i] = 256;
    }
    GDN_TRY(check_qk(fn, a, GDN_NORM_L2, 1, d, GDN_F32));
    *bytes = gdn::qk_norm_workspace_bytes(a);
    return ok();
}

gdn_status gdn_qk_norm_bwd(const void* q, const void* k, const void* grad_q_out, const void* grad_k_out,
                           const float* q_weight, const float* k_weight, gdn_norm norm, float eps, const float* cos,
                           const float* sin, int n_pos, int rotary_dim, int interleaved, const int32_t* positions,
                           void* grad_q, void* grad_k, float* grad_q_weight, float* grad_k_weight, int64_t n_tokens,
                           int T, int H_q, int H_k, int d, int64_t q_token_stride, int64_t q_head_stride,
                           int64_t k_token_stride, int64_t k_head_stride, gdn_dtype dtype, void* workspace,
                           size_t workspace_bytes, void* stream) {
    const char* fn = "gdn_qk_norm_bwd";
    gdn::QkNormArgs a{{q, k}, {grad_q_out, grad_k_out}, {grad_q, grad_k}, {q_weight, k_weight},
                      {grad_q_weight, grad_k_weight}, {q_token_stride, k_token_stride},
                      {q_head_stride, k_head_stride}, {H_q, H_k}, n_tokens, 0, 0, 0.f, eps, cos, sin, n_pos,
                      rotary_dim, interleaved != 0, positions, 0, nullptr};
    GDN_TRY(check_qk(fn, a, norm, T, d, dtype));
    const size_t es = size_of(dtype);
    if (a.n > 0) {
        GDN_TRY(need(fn, "grad_q_out", grad_q_out, es));
        GDN_TRY(need(fn, "grad_k_out", grad_k_out, es));
        GDN_TRY(need(fn, "grad_q", grad_q, es));
        GDN_TRY(need(fn, "grad_k", grad_k, es));
    }
    for (int i = 0; i < 2; ++i) {
        const char* name = i ? "grad_k_weight" : "grad_q_weight";
        if (a.w[i]) GDN_TRY(need(fn, name, a.dw[i], 4));
        else if (a.dw[i]) return fail(GDN_ERR_INVALID_ARG, "%s: %s is given without its weight", fn, name);
    }
    const size_t bytes = a.dw[0] || a.dw[1] ? gdn::qk_norm_workspace_bytes(a) : 0;     // (for the weights' gradients alone)
    Workspace ws;
    GDN_TRY(ws.get(fn, workspace, workspace_bytes, bytes, static_cast<cudaStream_t>(stream)));
    a.ws = ws.ptr;
    return finish(fn, gdn::launch_qk_norm_bwd(a, ws.s), ws);
}

gdn_status gdn_short_conv_fwd(const void* x, const float* weight, const float* bias, gdn_activation activation,
                              const void* initial_state, void* final_state, const int32_t* cu_seqlens, int n_seqs,
                              void* y, int B, int T, int D, int W, int64_t ld_x, gdn_dtype dtype, void* stream) {
    const char* fn = "gdn_short_conv_fwd";
    GDN_TRY(check_sizes(fn, B, T, D, cu_seqlens, n_seqs));
    GDN_TRY(check_conv(fn, activation, W, D, ld_x, dtype));
    const size_t es = size_of(dtype);
    if (T > 0) {
        GDN_TRY(need(fn, "x", x, es));
        GDN_TRY(need(fn, "y", y, es));
    }
    GDN_TRY(need(fn, "weight", weight, 4));
    GDN_TRY(may(fn, "bias", bias, 4));
    GDN_TRY(may(fn, "initial_state", initial_state, es));
    GDN_TRY(may(fn, "final_state", final_state, es));
    gdn::ConvArgs a{};
    a.x = x; a.w = weight; a.b = bias; a.silu = activation == GDN_ACT_SILU; a.h0 = initial_state; a.hT = final_state;
    a.cu = cu_seqlens; a.n_seqs = n_seqs; a.y = y; a.B = B; a.T = T; a.D = D; a.W = W; a.ldx = ld_x;
    a.bf16 = dtype == GDN_BF16;
    const cudaError_t e = gdn::launch_conv_fwd(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}

gdn_status gdn_short_conv_workspace_size(int B, int T, int D, int W, size_t* bytes) {
    const char* fn = "gdn_short_conv_workspace_size";
    if (!bytes) return fail(GDN_ERR_INVALID_ARG, "%s: bytes is NULL", fn);
    GDN_TRY(check_sizes(fn, B, T, D, nullptr, 0));
    GDN_TRY(check_conv(fn, GDN_ACT_NONE, W, D, D, GDN_F32));
    gdn::ConvArgs a{};
    a.B = B; a.T = T; a.D = D; a.W = W;
    *bytes = gdn::conv_workspace_bytes(a);
    return ok();
}

gdn_status gdn_short_conv_bwd(const void* x, const float* weight, const float* bias, gdn_activation activation,
                              const void* initial_state, const void* grad_y, const void* grad_final_state,
                              const int32_t* cu_seqlens, int n_seqs, void* grad_x, float* grad_weight,
                              float* grad_bias, void* grad_initial_state, int B, int T, int D, int W, int64_t ld_x,
                              gdn_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "gdn_short_conv_bwd";
    GDN_TRY(check_sizes(fn, B, T, D, cu_seqlens, n_seqs));
    GDN_TRY(check_conv(fn, activation, W, D, ld_x, dtype));
    const size_t es = size_of(dtype);
    if (T > 0) {
        GDN_TRY(need(fn, "x", x, es));
        GDN_TRY(need(fn, "grad_y", grad_y, es));
        GDN_TRY(need(fn, "grad_x", grad_x, es));
    }
    GDN_TRY(need(fn, "weight", weight, 4));
    GDN_TRY(need(fn, "grad_weight", grad_weight, 4));
    GDN_TRY(may(fn, "bias", bias, 4));
    if (grad_bias && !bias) return fail(GDN_ERR_INVALID_ARG, "%s: grad_bias is given without bias", fn);
    GDN_TRY(may(fn, "grad_bias", grad_bias, 4));
    GDN_TRY(may(fn, "initial_state", initial_state, es));
    GDN_TRY(may(fn, "grad_final_state", grad_final_state, es));
    GDN_TRY(may(fn, "grad_initial_state", grad_initial_state, es));
    gdn::ConvArgs a{};
    a.x = x; a.w = weight; a.b = bias; a.silu = activation == GDN_ACT_SILU; a.h0 = initial_state;
    a.cu = cu_seqlens; a.n_seqs = n_seqs; a.dy = grad_y; a.dhT = grad_final_state; a.dx = grad_x; a.dw = grad_weight;
    a.db = grad_bias; a.dh0 = grad_initial_state; a.B = B; a.T = T; a.D = D; a.W = W; a.ldx = ld_x;
    a.bf16 = dtype == GDN_BF16;
    Workspace ws;
    GDN_TRY(ws.get(fn, workspace, workspace_bytes, gdn::conv_workspace_bytes(a), static_cast<cudaStream_t>(stream)));
    a.ws = ws.ptr;
    return finish(fn, gdn::launch_conv_bwd(a, ws.s), ws);
}

gdn_status gdn_short_conv_step(const void* x, const float* weight, const float* bias, gdn_activation activation,
                               const void* state, void* state_out, void* y, int N, int D, int W, int64_t ld_x,
                               gdn_dtype dtype, void* stream) {
    const char* fn = "gdn_short_conv_step";
    GDN_TRY(check_sizes(fn, N, 1, D, nullptr, 0));
    GDN_TRY(check_conv(fn, activation, W, D, ld_x, dtype));
    const size_t es = size_of(dtype);
    GDN_TRY(need(fn, "x", x, es));
    GDN_TRY(need(fn, "weight", weight, 4));
    GDN_TRY(may(fn, "bias", bias, 4));
    GDN_TRY(need(fn, "state", state, es));
    GDN_TRY(need(fn, "state_out", state_out, es));
    GDN_TRY(need(fn, "y", y, es));
    gdn::ConvArgs a{};
    a.x = x; a.w = weight; a.b = bias; a.silu = activation == GDN_ACT_SILU; a.y = y; a.B = N; a.T = 1; a.D = D;
    a.W = W; a.ldx = ld_x; a.bf16 = dtype == GDN_BF16;
    const cudaError_t e = gdn::launch_conv_step(a, state, state_out, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}

}  // extern "C"
