"""The 64-bit references of the operators around the delta rule: their gradients against central differences of their
forwards (step 1e-5, so the truncation error is about 1e-10 and the rounding error about 1e-10 of the sums: tolerance
1e-7 relative to the largest gradient), and closed forms.
"""
import numpy as np
import pytest

import mixer_reference as R

STEP, TOL = 1e-5, 1e-7


def _differences(loss, arrays, grads):
    rng = np.random.default_rng(0)
    for name, x in arrays.items():
        g = grads[name]
        scale = max(1.0, np.abs(g).max())
        for flat in rng.choice(x.size, size=min(x.size, 24), replace=False):
            at = np.unravel_index(flat, x.shape)
            keep = x[at]
            x[at] = keep + STEP
            up = loss()
            x[at] = keep - STEP
            down = loss()
            x[at] = keep
            assert abs((up - down) / (2 * STEP) - g[at]) <= TOL * scale, (name, at)


@pytest.mark.parametrize("cu", [None, [0, 4, 4, 9]])
@pytest.mark.parametrize("act,gate,normalize", [(False, False, False), (True, True, True), (True, False, True),
                                                (False, True, True)])
def test_recurrence_gradients(cu, act, gate, normalize):
    rng = np.random.default_rng(1)
    B, T, D = (2, 9, 3) if cu is None else (1, 9, 3)
    N = B if cu is None else 3
    x, do = rng.normal(size=(2, B, T, D))
    g = rng.normal(size=(B, T, D)) if act else -np.exp(rng.normal(size=(B, T, D)) - 1)
    i = rng.normal(size=(B, T, D)) if gate else None
    A = rng.normal(size=D) * 0.5 if act else None
    dt = rng.normal(size=D) if act else None
    h0, dhT = rng.normal(size=(2, N, D))
    kw = dict(i=i, A_log=A, dt_bias=dt, normalize=normalize, h0=h0, cu=cu)
    grads = R.glr_bwd(x, g, do, dhT, **kw)

    def loss():
        o, hT, _ = R.glr_fwd(x, g, **kw)
        return (o * do).sum() + (hT * dhT).sum()
    arrays = {"dx": x, "dg": g, "dh0": h0}
    if gate:
        arrays["di"] = i
    if act:
        arrays.update(dA_log=A, ddt_bias=dt)
    _differences(loss, arrays, grads)


@pytest.mark.parametrize("l2", [False, True])
@pytest.mark.parametrize("rot,interleaved", [(0, False), (6, False), (4, True)])
def test_head_norm_gradients(l2, rot, interleaved):
    rng = np.random.default_rng(2)
    x, dz = rng.normal(size=(2, 3, 2, 7))
    w = rng.normal(size=7)
    cos = sin = None
    if rot:
        ang = rng.normal(size=(3, rot // 2))
        cos, sin = np.cos(ang), np.sin(ang)
    dx, dw, _, _ = R.head_norm_bwd(x, w, l2, 1e-6, cos, sin, interleaved, dz)
    _differences(lambda: (R.head_norm_fwd(x, w, l2, 1e-6, cos, sin, interleaved) * dz).sum(), {"x": x, "w": w},
                 {"x": dx, "w": dw})


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("cu", [None, [0, 1, 1, 3, 9]])
@pytest.mark.parametrize("silu", [True, False])
def test_convolution_gradients(W, cu, silu):
    rng = np.random.default_rng(3)
    B, T, D = (2, 5, 3) if cu is None else (1, 9, 3)
    N = B if cu is None else 4
    x, dy = rng.normal(size=(2, B, T, D))
    w, b = rng.normal(size=(D, W)), rng.normal(size=D)
    h0, dhT = rng.normal(size=(2, N, W - 1, D))
    grads = R.conv_bwd(x, w, dy, b, silu, h0, dhT, cu)

    def loss():
        y, hT = R.conv_fwd(x, w, b, silu, h0, cu)
        return (y * dy).sum() + (hT * dhT).sum()
    _differences(loss, {"dx": x, "dw": w, "db": b, "dh0": h0}, grads)


def test_closed_forms():
    # a = 1: a running sum; a = 0: no memory; a constant decay of a constant input: the geometric sum
    x = np.random.default_rng(4).normal(size=(1, 6, 2))
    o, _, _ = R.glr_fwd(x, np.zeros_like(x))
    assert np.allclose(o, np.cumsum(x, 1), rtol=0, atol=1e-15 * 6)
    with np.errstate(divide="ignore"):
        o, _, _ = R.glr_fwd(x, np.log(np.zeros_like(x)))
    assert np.array_equal(o, x)
    o, _, _ = R.glr_fwd(np.ones((1, 5, 1)), np.full((1, 5, 1), np.log(0.5)))
    assert np.allclose(o[0, :, 0], [1, 1.5, 1.75, 1.875, 1.9375])
    # the convolution with its last tap alone is the identity; with the one before, a shift
    w = np.zeros((2, 3))
    w[:, 2] = 1
    assert np.array_equal(R.conv_fwd(x, w, silu=False)[0], x)
    w = np.roll(w, -1, 1)
    assert np.array_equal(R.conv_fwd(x, w, silu=False)[0][:, 1:], x[:, :-1])
    # a unit-norm head keeps its length under the rotation
    y = R.head_norm_fwd(x[:, :, None], None, True, 0.0, np.cos(x[..., :1]), np.sin(x[..., :1]), True)
    assert np.allclose((y * y).sum(-1), 1)
