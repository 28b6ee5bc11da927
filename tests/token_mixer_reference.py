"""Linear attention with a decay for each head, and the paged cache's operators, in 64 bits, written from their formulas with
numpy.  test_token_mixer_reference.py checks the gradients against differences of the forward."""
import numpy as np

from mixer_reference import f64, spans  # noqa: F401  (f64: used by the tests)


def _heads(x, H):
    return np.repeat(x, H // x.shape[-2], axis=-2)


def lin_fwd(q, k, v, g, scale, h0=None, cu=None):
    """(o [B, T, H, dv], final states [N, H, dk, dv], and per sequence the states before its tokens [len, H, dk, dv])."""
    B, T, H, dv = v.shape
    q, k, g = _heads(q, H), _heads(k, H), np.broadcast_to(g, (B, T, H))
    sp = spans(B, T, cu)
    hT = np.zeros((len(sp), H, q.shape[-1], dv)) if h0 is None else h0.copy()
    o, before = np.zeros_like(v), []
    for n, b, lo, hi in sp:
        S, prev = hT[n], np.zeros((hi - lo,) + hT.shape[1:])
        for t in range(lo, hi):
            prev[t - lo] = S
            S = np.exp(g[b, t])[:, None, None] * S + k[b, t, :, :, None] * v[b, t, :, None, :]
            o[b, t] = scale * np.einsum("hk,hkv->hv", q[b, t], S)
        hT[n] = S
        before.append(prev)
    return o, hT, before


def lin_bwd(q, k, v, g, do, scale, h0=None, dhT=None, cu=None):
    """(dq, dk, dv, dg, dh0) of sum <do, o> + sum <dhT, final states>; dg has g's shape."""
    B, T, H, dv_ = v.shape
    Hk = q.shape[-2]
    _, hT, before = lin_fwd(q, k, v, g, scale, h0, cu)
    qh, kh, gh = _heads(q, H), _heads(k, H), np.broadcast_to(g, (B, T, H))
    dq, dk, dv, dg = np.zeros_like(qh), np.zeros_like(kh), np.zeros_like(v), np.zeros((B, T, H))
    dh0 = np.zeros_like(hT) if dhT is None else dhT.copy()
    for n, b, lo, hi in spans(B, T, cu):
        D = dh0[n]
        for t in range(hi - 1, lo - 1, -1):
            a = np.exp(gh[b, t])[:, None, None]
            S = a * before[n][t - lo] + kh[b, t, :, :, None] * v[b, t, :, None, :]
            D = D + scale * qh[b, t, :, :, None] * do[b, t, :, None, :]
            dq[b, t] = scale * np.einsum("hkv,hv->hk", S, do[b, t])
            dk[b, t] = np.einsum("hkv,hv->hk", D, v[b, t])
            dv[b, t] = np.einsum("hkv,hk->hv", D, kh[b, t])
            D = a * D
            dg[b, t] = (D * before[n][t - lo]).sum((-1, -2))
        dh0[n] = D
    dq, dk = (x.reshape(B, T, Hk, H // Hk, -1).sum(3) for x in (dq, dk))
    return dq, dk, dv, dg.sum((0, 1)) if np.ndim(g) == 1 else dg, dh0


def turn(x, cos, sin, interleaved):
    """Rotate the channels of [n, heads, d] by angles whose cosines and sines are [n, R / 2]."""
    R = 2 * cos.shape[-1]
    y = x.copy()
    i, j = (np.arange(0, R, 2), np.arange(1, R, 2)) if interleaved else (np.arange(R // 2), np.arange(R // 2, R))
    c, s = cos[:, None], sin[:, None]
    y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., j] * c + x[..., i] * s
    return y


def places(lengths, table, page_size, n_pages, n_tokens, cu=None):
    """(token, position, page, slot) of every new token; page None where it has none."""
    out = []
    for n, length in enumerate(lengths):
        lo, hi = (n, n + 1) if cu is None else (int(cu[n]), int(cu[n + 1]))
        for t in range(lo, hi):
            pos = int(length) - (hi - t)
            page = None
            if 0 <= pos < table.shape[1] * page_size:
                page = int(table[n, pos // page_size])
                page = page if 0 <= page < n_pages else None
            out.append((t, pos, page, pos % page_size))
    return out


def attn(q, kc, vc, table, lengths, scale):
    """(o [N, Hq, d], lse [N, Hq])."""
    N, Hq, d = q.shape
    n_pages, page, Hk, _ = kc.shape
    o, lse = np.zeros_like(q), np.full((N, Hq), -np.inf)
    for n in range(N):
        t = np.arange(min(max(int(lengths[n]), 0), table.shape[1] * page))
        pages = table[n, t // page]
        t, pages = t[(pages >= 0) & (pages < n_pages)], pages[(pages >= 0) & (pages < n_pages)]
        if len(t) == 0:
            continue
        k, v = (np.repeat(c[pages, t % page], Hq // Hk, axis=1) for c in (kc, vc))       # [L, Hq, d]
        s = scale * np.einsum("hd,lhd->hl", q[n], k)
        top = s.max(-1, keepdims=True)
        p = np.exp(s - top)
        o[n] = np.einsum("hl,lhd->hd", p, v) / p.sum(-1, keepdims=True)
        lse[n] = top[:, 0] + np.log(p.sum(-1))
    return o, lse
