"""The operators around the delta rule in 64 bits, written from their formulas with numpy, one token at a time.

Forward and hand-derived gradients of the gated linear recurrence, the query/key head norm with rotation, and the
short convolution.  test_mixer_reference.py checks the gradients against differences of the forwards.
"""
import numpy as np


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def spans(B, T, cu):
    """(sequence, batch row, first token, one past the last)."""
    if cu is None:
        return [(n, n, 0, T) for n in range(B)]
    cu = [int(v) for v in cu]
    return [(n, 0, cu[n], cu[n + 1]) for n in range(len(cu) - 1)]


def sigmoid(z):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-z))


# ------------------------------------------------------------------------------------------- gated linear recurrence

def _gates(x, g, i, A_log, dt_bias, normalize):
    z = g if dt_bias is None else g + dt_bias
    with np.errstate(over="ignore", invalid="ignore"):
        la = g if A_log is None else -np.exp(A_log) * np.logaddexp(0, z)
        a = np.exp(la)
        s = np.sqrt(np.maximum(-np.expm1(2 * la), 0)) if normalize else np.ones_like(a)
    si = np.ones_like(a) if i is None else sigmoid(i)
    return z, la, a, s, si


def glr_fwd(x, g, i=None, A_log=None, dt_bias=None, normalize=False, h0=None, cu=None):
    """(o [B, T, D], final states [N, D], states before every token)."""
    B, T, D = x.shape
    sp = spans(B, T, cu)
    _, _, a, s, si = _gates(x, g, i, A_log, dt_bias, normalize)
    h = np.zeros((len(sp), D)) if h0 is None else h0.copy()
    o, prev = np.zeros_like(x), np.zeros_like(x)
    for n, b, lo, hi in sp:
        for t in range(lo, hi):
            prev[b, t] = h[n]
            h[n] = a[b, t] * h[n] + s[b, t] * si[b, t] * x[b, t]
            o[b, t] = h[n]
    return o, h, prev


def glr_bwd(x, g, do, dhT=None, i=None, A_log=None, dt_bias=None, normalize=False, h0=None, cu=None):
    """dict of gradients, and "abs": the sums of magnitudes behind dA_log and ddt_bias."""
    B, T, D = x.shape
    sp = spans(B, T, cu)
    z, la, a, s, si = _gates(x, g, i, A_log, dt_bias, normalize)
    _, _, prev = glr_fwd(x, g, i, A_log, dt_bias, normalize, h0, cu)
    dh0 = np.zeros((len(sp), D)) if dhT is None else dhT.copy()
    dh = np.zeros_like(x)
    for n, b, lo, hi in sp:
        for t in range(hi - 1, lo - 1, -1):
            dh[b, t] = do[b, t] + dh0[n]
            dh0[n] = a[b, t] * dh[b, t]
    dla = a * dh * prev
    if normalize:
        with np.errstate(divide="ignore", invalid="ignore"):
            dla = dla - np.where(s > 0, dh * si * x * a * a / s, 0.0)
    out = {"dx": dh * s * si, "di": None if i is None else dh * s * x * si * (1 - si), "dh0": dh0, "dA_log": None,
           "ddt_bias": None, "dg": dla}
    if A_log is not None:
        dz = -dla * np.exp(A_log) * sigmoid(z)
        with np.errstate(invalid="ignore"):
            tA = np.where(dla == 0, 0.0, dla * la)
        out.update(dg=dz, dA_log=tA.sum((0, 1)), ddt_bias=dz.sum((0, 1)),
                   abs={"dA_log": np.abs(tA).sum((0, 1)), "ddt_bias": np.abs(dz).sum((0, 1))})
    return out


# --------------------------------------------------------------------------------------------- query/key head norm

def rotate(y, cos, sin, interleaved):
    """y [..., H, d]; cos, sin [..., rot / 2]."""
    if cos is None:
        return y
    half = cos.shape[-1]
    y = y.copy()
    i = np.arange(half) * 2 if interleaved else np.arange(half)
    j = i + 1 if interleaved else i + half
    c, s = cos[..., None, :], sin[..., None, :]
    y[..., i], y[..., j] = y[..., i] * c - y[..., j] * s, y[..., j] * c + y[..., i] * s
    return y


def head_norm_fwd(x, w, l2, eps, cos, sin, interleaved):
    m = (x * x).sum(-1, keepdims=True) if l2 else (x * x).mean(-1, keepdims=True)
    y = x / np.sqrt(m + eps)
    return rotate(y if w is None else y * w, cos, sin, interleaved)


def head_norm_bwd(x, w, l2, eps, cos, sin, interleaved, dz):
    """(dx, dw, the sums of magnitudes behind dw, the largest magnitude that dx is a difference of)."""
    c = 1.0 if l2 else 1.0 / x.shape[-1]
    r = 1 / np.sqrt(c * (x * x).sum(-1, keepdims=True) + eps)
    dy = rotate(dz, cos, None if sin is None else -sin, interleaved)
    e = dy if w is None else dy * w
    dx = r * (e - c * r * r * x * (x * e).sum(-1, keepdims=True))
    t = (dy * x * r).reshape(-1, x.shape[-1])
    return dx, t.sum(0), np.abs(t).sum(0), np.abs(r * e).max(initial=0.0)


# ----------------------------------------------------------------------------------------------- short convolution

def _padded(x, h0, W, n, b, lo, hi):
    first = np.zeros((W - 1, x.shape[-1])) if h0 is None else h0[n]
    return np.concatenate([first, x[b, lo:hi]])


def conv_fwd(x, w, b=None, silu=True, h0=None, cu=None):
    """(y, final states)."""
    B, T, D = x.shape
    W = w.shape[1]
    sp = spans(B, T, cu)
    y, hT = np.zeros_like(x), np.zeros((len(sp), W - 1, D))
    for n, r, lo, hi in sp:
        f = _padded(x, h0, W, n, r, lo, hi)
        for t in range(hi - lo):
            p = (f[t:t + W] * w.T).sum(0) + (0 if b is None else b)
            y[r, lo + t] = p * sigmoid(p) if silu else p
        hT[n] = f[hi - lo:]
    return y, hT


def conv_bwd(x, w, dy, b=None, silu=True, h0=None, dhT=None, cu=None):
    B, T, D = x.shape
    W = w.shape[1]
    sp = spans(B, T, cu)
    out = {"dx": np.zeros_like(x), "dw": np.zeros_like(w), "db": np.zeros(D), "dh0": np.zeros((len(sp), W - 1, D)),
           "abs": {"dw": np.zeros_like(w), "db": np.zeros(D)}}
    for n, r, lo, hi in sp:
        f = _padded(x, h0, W, n, r, lo, hi)
        df = np.zeros_like(f)
        if dhT is not None:
            df[hi - lo:] += dhT[n]
        for t in range(hi - lo):
            p = (f[t:t + W] * w.T).sum(0) + (0 if b is None else b)
            s = sigmoid(p)
            ds = dy[r, lo + t] * (s * (1 + p * (1 - s)) if silu else 1.0)
            df[t:t + W] += ds * w.T
            out["dw"] += (ds * f[t:t + W]).T
            out["db"] += ds
            out["abs"]["dw"] += np.abs(ds * f[t:t + W]).T
            out["abs"]["db"] += np.abs(ds)
        out["dh0"][n], out["dx"][r, lo:hi] = df[:W - 1], df[W - 1:]
    return out
