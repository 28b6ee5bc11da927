"""Argument checks of the operators around the delta rule, at the C ABI and in the binding.

Every call here is refused (or answered from its sizes alone) before any CUDA work: no GPU is needed.
"""
import ctypes

import pytest
import torch

import gated_delta_rule_gdn_gb300 as gdn
from gated_delta_rule_gdn_gb300 import _binding, _mixer, build

FAKE = 0x10000   # an aligned, never-dereferenced address: every call below fails validation first
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gdn.load()


def _call(f, a, kw):
    a = dict(a)
    assert set(kw) <= set(a), kw
    a.update(kw)
    return f(*a.values())


GLR = dict(x=FAKE, g=FAKE, i=FAKE, A=FAKE, dt=FAKE, norm=1, h0=FAKE)
GLR_TAIL = dict(B=2, T=64, D=32, ldx=32, ldg=32, ldi=32, dtype=1, gdtype=1, ws=FAKE, wsb=1 << 40, stream=None)
GLR_FWD = dict(GLR, hT=FAKE, cu=None, n=0, o=FAKE, ck=FAKE, **GLR_TAIL)
GLR_BWD = dict(GLR, do=FAKE, dhT=FAKE, cu=None, n=0, ck=FAKE, dx=FAKE, dg=FAKE, di=FAKE, dh0=FAKE, dA=FAKE, ddt=FAKE,
               **GLR_TAIL)
GLR_BAD = [
    (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(D=0), INVALID), (dict(dtype=3), INVALID), (dict(gdtype=2), INVALID),
    (dict(dtype=0, gdtype=1), UNSUPPORTED), (dict(x=None), INVALID), (dict(g=None), INVALID), (dict(x=FAKE + 1), INVALID),
    (dict(i=FAKE + 1), INVALID), (dict(A=None), INVALID), (dict(A=FAKE + 2), INVALID), (dict(dt=FAKE + 2), INVALID),
    (dict(h0=FAKE + 2), INVALID), (dict(ldx=31), INVALID), (dict(ldg=0), INVALID), (dict(ldi=-32), INVALID),
    (dict(ldx=1 << 32), INVALID), (dict(cu=FAKE, n=2), INVALID), (dict(B=1, cu=FAKE, n=0), INVALID),
    (dict(B=1, cu=FAKE + 2, n=1), INVALID), (dict(B=1 << 16, T=1 << 16), UNSUPPORTED),
    (dict(B=1, T=1 << 30, D=1 << 20, ldx=1 << 20, ldg=1 << 20, ldi=1 << 20), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", GLR_BAD + [(dict(o=None), INVALID), (dict(o=FAKE + 1), INVALID),
                                                 (dict(hT=FAKE + 1), INVALID), (dict(ck=FAKE + 2), INVALID)])
def test_scan_forward(lib, kw, status):
    assert _call(lib.glr_scan_fwd, GLR_FWD, kw) == status
    assert "glr_scan_fwd" in _binding.last_error()


@pytest.mark.parametrize("kw,status", GLR_BAD + [
    (dict(do=None), INVALID), (dict(dx=None), INVALID), (dict(dg=None), INVALID), (dict(di=None), INVALID),
    (dict(dA=None), INVALID), (dict(dt=None), INVALID), (dict(dhT=FAKE + 1), INVALID), (dict(dh0=FAKE + 2), INVALID),
    (dict(wsb=16), INVALID), (dict(ws=FAKE + 16), INVALID)])
def test_scan_backward(lib, kw, status):
    assert _call(lib.glr_scan_bwd, GLR_BWD, kw) == status
    assert "glr_scan_bwd" in _binding.last_error()


STEP = dict(GLR, hout=FAKE, o=FAKE, N=2, D=32, ldx=32, ldg=32, ldi=32, dtype=1, gdtype=1, stream=None)


@pytest.mark.parametrize("kw", [dict(N=0), dict(D=0), dict(h0=None), dict(hout=None), dict(o=None), dict(x=FAKE + 1),
                                dict(hout=FAKE + 2), dict(ldx=31), dict(A=None), dict(dtype=9)])
def test_scan_step(lib, kw):
    assert _call(lib.glr_step, STEP, kw) == INVALID
    assert "glr_step" in _binding.last_error()


QK_MID = dict(wq=FAKE, wk=FAKE, norm=0, eps=1e-6, cos=FAKE, sin=FAKE, P=100, rot=64, inter=0, pos=None)
QK_TAIL = dict(n=10, T=10, Hq=4, Hk=2, d=128, qt=512, qh=128, kt=256, kh=128, dtype=1)
QK_FWD = dict(q=FAKE, k=FAKE, **QK_MID, qo=FAKE, ko=FAKE, **QK_TAIL, stream=None)
QK_BWD = dict(q=FAKE, k=FAKE, dqo=FAKE, dko=FAKE, **QK_MID, dq=FAKE, dk=FAKE, dwq=FAKE, dwk=FAKE, **QK_TAIL, ws=FAKE,
              wsb=1 << 40, stream=None)
QK_BAD = [
    (dict(q=None), INVALID), (dict(k=FAKE + 1), INVALID), (dict(norm=2), INVALID), (dict(eps=0.0), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(rot=63), INVALID), (dict(rot=130), INVALID), (dict(rot=-2), INVALID), (dict(cos=None), INVALID),
    (dict(sin=FAKE + 2), INVALID), (dict(P=0), INVALID), (dict(P=9), INVALID), (dict(pos=FAKE + 2), INVALID),
    (dict(wq=FAKE + 1), INVALID), (dict(n=-1), INVALID), (dict(T=0), INVALID), (dict(Hq=0), INVALID), (dict(Hk=0), INVALID),
    (dict(d=0), UNSUPPORTED), (dict(d=257, qh=257, kh=257), UNSUPPORTED), (dict(qh=127), INVALID), (dict(kt=64), INVALID),
    (dict(dtype=5), INVALID), (dict(n=1 << 30), UNSUPPORTED), (dict(qt=1 << 33), INVALID),
]


@pytest.mark.parametrize("kw,status", QK_BAD + [(dict(qo=None), INVALID), (dict(ko=FAKE + 1), INVALID)])
def test_head_norm_forward(lib, kw, status):
    assert _call(lib.gdn_qk_norm_fwd, QK_FWD, kw) == status
    assert "gdn_qk_norm_fwd" in _binding.last_error()


@pytest.mark.parametrize("kw,status", QK_BAD + [
    (dict(dqo=None), INVALID), (dict(dk=None), INVALID), (dict(dwq=None), INVALID), (dict(wk=None), INVALID),
    (dict(wsb=8), INVALID), (dict(ws=FAKE + 64), INVALID)])
def test_head_norm_backward(lib, kw, status):
    assert _call(lib.gdn_qk_norm_bwd, QK_BWD, kw) == status
    assert "gdn_qk_norm_bwd" in _binding.last_error()


CONV_FWD = dict(x=FAKE, w=FAKE, b=FAKE, act=1, h0=FAKE, hT=FAKE, cu=None, n=0, y=FAKE, B=2, T=9, D=16, W=4, ldx=16, dtype=1,
                stream=None)
CONV_BWD = dict(x=FAKE, w=FAKE, b=FAKE, act=1, h0=FAKE, dy=FAKE, dhT=FAKE, cu=None, n=0, dx=FAKE, dw=FAKE, db=FAKE, dh0=FAKE,
                B=2, T=9, D=16, W=4, ldx=16, dtype=1, ws=FAKE, wsb=1 << 40, stream=None)
CONV_STEP = dict(x=FAKE, w=FAKE, b=FAKE, act=1, h=FAKE, hout=FAKE, y=FAKE, N=2, D=16, W=4, ldx=16, dtype=1, stream=None)
CONV_BAD = [
    (dict(x=None), INVALID), (dict(x=FAKE + 1), INVALID), (dict(w=None), INVALID), (dict(w=FAKE + 2), INVALID),
    (dict(b=FAKE + 1), INVALID), (dict(act=2), INVALID), (dict(act=-1), INVALID), (dict(W=1), UNSUPPORTED),
    (dict(W=5), UNSUPPORTED), (dict(D=0), INVALID), (dict(ldx=15), INVALID), (dict(dtype=4), INVALID),
]
CONV_SEQ = [(dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(h0=FAKE + 1), INVALID), (dict(cu=FAKE, n=1), INVALID),
            (dict(B=1, cu=FAKE, n=0), INVALID)]


@pytest.mark.parametrize("kw,status", CONV_BAD + CONV_SEQ + [(dict(y=None), INVALID), (dict(hT=FAKE + 1), INVALID)])
def test_convolution_forward(lib, kw, status):
    assert _call(lib.gdn_short_conv_fwd, CONV_FWD, kw) == status
    assert "gdn_short_conv_fwd" in _binding.last_error()


@pytest.mark.parametrize("kw,status", CONV_BAD + CONV_SEQ + [
    (dict(dy=None), INVALID), (dict(dx=FAKE + 1), INVALID), (dict(dw=None), INVALID), (dict(b=None), INVALID),
    (dict(dhT=FAKE + 1), INVALID), (dict(dh0=FAKE + 1), INVALID), (dict(wsb=8), INVALID), (dict(ws=FAKE + 128), INVALID)])
def test_convolution_backward(lib, kw, status):
    assert _call(lib.gdn_short_conv_bwd, CONV_BWD, kw) == status
    assert "gdn_short_conv_bwd" in _binding.last_error()


@pytest.mark.parametrize("kw,status", CONV_BAD + [(dict(h=None), INVALID), (dict(hout=None), INVALID), (dict(y=None), INVALID),
                                                  (dict(N=0), INVALID), (dict(h=FAKE + 1), INVALID)])
def test_convolution_step(lib, kw, status):
    assert _call(lib.gdn_short_conv_step, CONV_STEP, kw) == status
    assert "gdn_short_conv_step" in _binding.last_error()


def test_workspace_sizes(lib):
    assert gdn.glr_workspace_size(1, 0, 8) >= 0
    # the backward can compute its checkpoints itself: a state per 64 tokens of every row
    assert gdn.glr_workspace_size(2, 1000, 100, backward=True) >= 2 * 16 * 100 * 4
    assert gdn.qk_norm_workspace_size(1000, 4, 2, 128) > 0
    assert gdn.short_conv_workspace_size(2, 1000, 64, 4) > 0
    for bad in (lambda: gdn.glr_workspace_size(0, 1, 8), lambda: gdn.glr_workspace_size(1, 1, 8, -1),
                lambda: gdn.qk_norm_workspace_size(-1, 1, 1, 8), lambda: gdn.short_conv_workspace_size(1, 1, 8, 9)):
        with pytest.raises(gdn.GdnError):
            bad()
    for f, args in ((lib.glr_workspace_size, (0, 1, 1, 1, 0)), (lib.gdn_qk_norm_workspace_size, (1, 1, 1, 8)),
                    (lib.gdn_short_conv_workspace_size, (1, 1, 1, 4))):
        assert f(*args, None) == INVALID
        assert f(*args, ctypes.byref(ctypes.c_size_t())) == 0


def test_binding_refuses_wrong_tensors(lib):
    x = torch.zeros(1, 4, 8)
    for bad in (lambda: gdn.glr_scan_fwd(x, x), lambda: gdn.glr_scan_bwd(x, x, x), lambda: gdn.glr_step(x[0], x[0], x[0]),
                lambda: gdn.gdn_qk_norm_fwd(x, x), lambda: gdn.gdn_qk_norm_bwd(x, x, x, x),
                lambda: gdn.gdn_short_conv_fwd(x, torch.zeros(8, 4)), lambda: gdn.gdn_short_conv_bwd(x, torch.zeros(8, 4), x),
                lambda: gdn.gdn_short_conv_step(x[0], x, torch.zeros(8, 4)), lambda: gdn.glr_scan_fwd(x[0], x[0]),
                lambda: gdn.glr_scan_fwd(x.double(), x)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises((TypeError, ValueError)):
        gdn.glr_scan_fwd(None, x)


def test_row_spacing(lib):
    """The one row stride that a strided view has, or the refusal of a view that has none."""
    base = torch.zeros(4, 6, 20)
    rows = lambda t: _mixer.native().spacing(t)[0]     # noqa: E731
    assert rows(base) == 20
    assert rows(base[..., 3:11]) == 20
    assert rows(base[:, :1, :5]) == 120           # one token of every row
    assert rows(base[1:2, ::2, :5]) == 40
    assert rows(base[:1, :1, 2:3]) == 1           # a single row: its own width
    for bad in (base[..., ::2], base[:, :3, :5], base.transpose(0, 1), base[..., :1].expand(4, 6, 20),
                base[:, :1].expand(4, 6, 20)):
        with pytest.raises(ValueError):
            rows(bad)
    heads = lambda t: _mixer.native().spacing(t, heads=True)     # noqa: E731
    q = torch.zeros(4, 6, 10 * 16)[..., 32:96].unflatten(-1, (4, 16))
    assert heads(q) == (160, 16)
    assert heads(q[:, :, 1:2]) == (160, 16)       # a single head
    with pytest.raises(ValueError):
        heads(q.transpose(1, 2))
    with pytest.raises(ValueError):
        heads(q[..., :1, :].expand(4, 6, 4, 16))


def test_binding_arguments(lib):
    x = torch.zeros(1, 4, 8)
    for bad in (lambda: gdn.glr_scan_fwd(), lambda: gdn.glr_scan_fwd(x), lambda: gdn.glr_scan_fwd(x, x, what=1),
                lambda: gdn.glr_scan_fwd(x, x, x=x), lambda: gdn.glr_step(*([x] * 30)), lambda: gdn.glr_scan_fwd(3, x),
                lambda: _mixer.native().spacing(None)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(AttributeError):
        gdn.no_such_entry
    import inspect
    for name in _mixer.ENTRIES:
        assert name in gdn.__all__ and "stream" in inspect.signature(getattr(gdn, name)).parameters
