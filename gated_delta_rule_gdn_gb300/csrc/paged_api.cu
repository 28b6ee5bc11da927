// C ABI of the paged key-value cache (declared in include/gdn.h): argument checks and dispatch.

#include <cmath>

#include "internal.h"
#include "mixer_check.h"
#include "paged.h"

namespace {

gdn_status check_side(const char* fn, const char* name, const gdn_paged_side& x, size_t es, int d) {
    GDN_TRY(need(fn, name, x.data, es));
    const int64_t most = int64_t(1) << 40;
    if (x.page_stride < d || x.slot_stride < d || x.head_stride < d || x.page_stride > most || x.slot_stride > most || x.head_stride > most)
        return fail(GDN_ERR_INVALID_ARG, "%s: the page, slot and head strides of %s must be d..2^40 elements (got %lld, %lld, %lld)", fn,
                    name, (long long)x.page_stride, (long long)x.slot_stride, (long long)x.head_stride);
    return GDN_OK;
}

gdn_status check_cache(const char* fn, const gdn_paged_cache* p, int H_q, gdn::PagedCache& c) {
    if (!p) return fail(GDN_ERR_INVALID_ARG, "%s: cache must be non-NULL", fn);
    if (!dtype_ok(p->dtype)) return fail(GDN_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)p->dtype);
    if (p->N < 0 || p->n_pages < 0 || p->max_pages < 0 || p->page_size < 1 || p->H_k < 1 || p->d < 1)
        return fail(GDN_ERR_INVALID_ARG, "%s: need N, n_pages, max_pages >= 0 and page_size, H_k, d >= 1 (got %d, %d, %d, %d, %d, %d)",
                    fn, p->N, p->n_pages, p->max_pages, p->page_size, p->H_k, p->d);
    if (p->d > 256) return fail(GDN_ERR_UNSUPPORTED, "%s: the head size must be 1..256 (got %d)", fn, p->d);
    if (H_q < 0 || H_q % p->H_k)
        return fail(GDN_ERR_INVALID_ARG, "%s: H_q=%d query heads are no multiple of H_k=%d key heads", fn, H_q, p->H_k);
    if (p->N > (1 << 24) || (int64_t)p->N * (H_q > p->H_k ? H_q : p->H_k) > (1 << 24))
        return fail(GDN_ERR_UNSUPPORTED, "%s: sequences times heads is more than 2^24 (N=%d)", fn, p->N);
    if ((int64_t)p->max_pages * p->page_size > 0x7FFFFF00)
        return fail(GDN_ERR_UNSUPPORTED, "%s: max_pages * page_size is more than 2^31 - 256", fn);
    const size_t es = size_of(p->dtype);
    if (p->n_pages > 0) {
        GDN_TRY(check_side(fn, "k_cache", p->k, es, p->d));
        GDN_TRY(check_side(fn, "v_cache", p->v, es, p->d));
    }
    if (p->N > 0) {
        GDN_TRY(need(fn, "lengths", p->lengths, 4));
        if (p->max_pages > 0) GDN_TRY(need(fn, "block_table", p->block_table, 4));
        if (p->table_stride < p->max_pages)
            return fail(GDN_ERR_INVALID_ARG, "%s: the row stride of block_table must be max_pages or more (got %lld, %d)", fn,
                        (long long)p->table_stride, p->max_pages);
    }
    c.k = {p->k.data, p->k.page_stride, p->k.slot_stride, p->k.head_stride};
    c.v = {p->v.data, p->v.page_stride, p->v.slot_stride, p->v.head_stride};
    c.table = p->block_table;
    c.table_ld = p->table_stride;
    c.max_pages = p->max_pages;
    c.page_size = p->page_size;
    c.n_pages = p->n_pages;
    c.lengths = p->lengths;
    c.N = p->N;
    c.Hk = p->H_k;
    c.d = p->d;
    c.bf16 = p->dtype == GDN_BF16;
    return GDN_OK;
}

gdn_status check_strides(const char* fn, const char* name, int64_t tok, int64_t head, int d) {
    if (tok < d || head < d || tok > (int64_t(1) << 31) || head > (int64_t(1) << 31))
        return fail(GDN_ERR_INVALID_ARG, "%s: the token and head strides of %s must be %d..2^31 elements (got %lld, %lld)", fn, name, d,
                    (long long)tok, (long long)head);
    return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status paged_append(const void* k, const void* v, const void* q, const gdn_paged_cache* cache, const int32_t* cu_seqlens,
                        const float* cos, const float* sin, int n_pos, int rotary_dim, int interleaved, void* q_out,
                        int64_t n_tokens, int H_q, int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                        int64_t v_head_stride, int64_t q_token_stride, int64_t q_head_stride, void* stream) {
    const char* fn = "paged_append";
    gdn::PagedAppendArgs a{};
    GDN_TRY(check_cache(fn, cache, q ? H_q : 0, a.c));
    const int d = a.c.d;
    const size_t es = size_of(cache->dtype);
    if (n_tokens < 0 || n_tokens > kMaxRows)
        return fail(GDN_ERR_INVALID_ARG, "%s: n_tokens must be 0..%lld (got %lld)", fn, (long long)kMaxRows, (long long)n_tokens);
    if (!cu_seqlens && n_tokens != a.c.N)
        return fail(GDN_ERR_INVALID_ARG, "%s: without cu_seqlens each of the %d sequences has one new token (got %lld)", fn, a.c.N,
                    (long long)n_tokens);
    if (n_tokens > 0 && a.c.N < 1) return fail(GDN_ERR_INVALID_ARG, "%s: tokens are given without a sequence", fn);
    if (rotary_dim < 0 || rotary_dim > d || rotary_dim % 2)
        return fail(GDN_ERR_INVALID_ARG, "%s: rotary_dim must be even and 0..d (got %d, d=%d)", fn, rotary_dim, d);
    if (rotary_dim > 0) {
        GDN_TRY(need(fn, "cos", cos, 4));
        GDN_TRY(need(fn, "sin", sin, 4));
        if (n_pos < 1) return fail(GDN_ERR_INVALID_ARG, "%s: the rotation table needs n_pos >= 1 (got %d)", fn, n_pos);
    }
    GDN_TRY(may(fn, "cu_seqlens", cu_seqlens, 4));
    GDN_TRY(check_strides(fn, "k", k_token_stride, k_head_stride, d));
    GDN_TRY(check_strides(fn, "v", v_token_stride, v_head_stride, d));
    if (q) {
        if (H_q < 1) return fail(GDN_ERR_INVALID_ARG, "%s: q needs H_q >= 1 (got %d)", fn, H_q);
        GDN_TRY(need(fn, "q", q, es));
        GDN_TRY(check_strides(fn, "q", q_token_stride, q_head_stride, d));
        if (n_tokens > 0) GDN_TRY(need(fn, "q_out", q_out, es));
    }
    if (n_tokens == 0) return ok();
    GDN_TRY(need(fn, "k", k, es));
    GDN_TRY(need(fn, "v", v, es));
    a.k = k; a.v = v; a.q = q;
    a.k_tok = k_token_stride; a.k_head = k_head_stride; a.v_tok = v_token_stride; a.v_head = v_head_stride;
    a.q_tok = q_token_stride; a.q_head = q_head_stride;
    a.Hq = H_q; a.n_tokens = n_tokens; a.cu = cu_seqlens; a.cos = cos; a.sin = sin;
    a.n_pos = n_pos; a.rot = rotary_dim; a.interleaved = interleaved != 0; a.q_out = q_out;
    const cudaError_t e = gdn::launch_paged_append(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}

gdn_status paged_attn_workspace_size(int N, int H_q, int H_k, int d, int max_pages, int page_size, size_t* bytes) {
    const char* fn = "paged_attn_workspace_size";
    if (!bytes) return fail(GDN_ERR_INVALID_ARG, "%s: bytes is NULL", fn);
    gdn::PagedAttnArgs a{};
    gdn_paged_cache c{};
    c.N = N; c.H_k = H_k; c.d = d; c.max_pages = max_pages; c.page_size = page_size; c.table_stride = max_pages;
    c.block_table = c.lengths = reinterpret_cast<const int32_t*>(uintptr_t(1) << 20);
    GDN_TRY(check_cache(fn, &c, H_q, a.c));
    a.Hq = H_q;
    a.splits = gdn::paged_attn_splits(a);
    *bytes = gdn::paged_attn_workspace_bytes(a);
    return ok();
}

gdn_status paged_attn_step(const void* q, const gdn_paged_cache* cache, float scale, void* o, float* lse, int H_q,
                           int64_t q_token_stride, int64_t q_head_stride, void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "paged_attn_step";
    gdn::PagedAttnArgs a{};
    GDN_TRY(check_cache(fn, cache, H_q, a.c));
    if (H_q < 1) return fail(GDN_ERR_INVALID_ARG, "%s: need H_q >= 1 (got %d)", fn, H_q);
    const size_t es = size_of(cache->dtype);
    GDN_TRY(check_strides(fn, "q", q_token_stride, q_head_stride, a.c.d));
    if (a.c.N == 0) return ok();
    GDN_TRY(need(fn, "q", q, es));
    GDN_TRY(need(fn, "o", o, es));
    GDN_TRY(may(fn, "lse", lse, 4));
    if (a.c.n_pages == 0) a.c.k.p = a.c.v.p = const_cast<void*>(q);      // (nothing is read, but copies of no bytes have an address)
    a.q = q; a.q_tok = q_token_stride; a.q_head = q_head_stride; a.Hq = H_q; a.scale = scale; a.o = o; a.lse = lse;
    a.splits = gdn::paged_attn_splits(a);
    if ((int64_t)a.c.N * H_q * a.splits > (int64_t(1) << 31) - 1)
        return fail(GDN_ERR_UNSUPPORTED, "%s: N=%d, H_q=%d and %d parts need more than 2^31 blocks", fn, a.c.N, H_q, a.splits);
    Workspace ws;
    GDN_TRY(ws.get(fn, workspace, workspace_bytes, gdn::paged_attn_workspace_bytes(a), static_cast<cudaStream_t>(stream)));
    a.ws = ws.ptr;
    return finish(fn, gdn::launch_paged_attn(a, ws.s), ws);
}

}  // extern "C"
