"""The short convolution in 64 bits over many tokens at once: every sequence is laid out behind its initial state, and the
taps are whole-array shifts.  (mixer_reference.py has it token by token; test_mixer_host.py compares the two.)
"""
import numpy as np

from mixer_reference import sigmoid


def conv(x, w, dy=None, b=None, silu=True, h0=None, dhT=None, cu=None):
    """dict of y, hT, and with dy the gradients; "abs": the sums of magnitudes behind dw and db."""
    B, T, D = x.shape
    W = w.shape[1]
    cu = np.arange(0, B * T + 1, T) if cu is None else np.asarray(cu)
    N, lens = len(cu) - 1, np.diff(cu)
    seq = np.repeat(np.arange(N), lens)
    at = np.arange(B * T) + (seq + 1) * (W - 1)                 # a token's place, and the first of a sequence's state
    head = cu[:-1] + np.arange(N) * (W - 1)
    states, tail = head[:, None] + np.arange(W - 1), (head + lens)[:, None] + np.arange(W - 1)
    f = np.zeros((B * T + N * (W - 1), D))
    f[at] = x.reshape(-1, D)
    if h0 is not None:
        f[states] = h0
    p = sum(w[:, j] * f[at - (W - 1) + j] for j in range(W)) + (0 if b is None else b)
    s = sigmoid(p)
    out = {"y": (p * s if silu else p).reshape(x.shape), "hT": f[tail]}
    if dy is None:
        return out
    ds = dy.reshape(-1, D) * (s * (1 + p * (1 - s)) if silu else 1.0)
    df = np.zeros_like(f)
    if dhT is not None:
        df[tail] += dhT
    terms = [ds * f[at - (W - 1) + j] for j in range(W)]
    for j in range(W):
        df[at - (W - 1) + j] += ds * w[:, j]
    out.update(dx=df[at].reshape(x.shape), dh0=df[states], dw=np.stack([t.sum(0) for t in terms], 1), db=ds.sum(0),
               abs={"dw": np.stack([np.abs(t).sum(0) for t in terms], 1), "db": np.abs(ds).sum(0)})
    return out
