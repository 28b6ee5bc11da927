"""GPU parity of the operators around the delta rule (gated linear recurrence, query/key head norm with rotation, short
convolution) against their 64-bit references.

Tolerances, from the arithmetic:
* An fp32 result of the recurrence gathers one rounding of 2^-24 and a decay off by a few units for every token in its
  memory; signs are mixed, so the 2-norm grows like the root of the length: rel-L2 <= 2^-22 (8 + sqrt T), and an
  element is off by at most the linear law, 2^-22 (8 + T) of the largest one.  A gradient multiplies up to four such
  factors: four times that.
* Results rounded to bf16 (8 significant bits) add the unit roundoff 2^-8 of the element, and so of the 2-norm.
* fp32 underflows below 2^-126.
* The norm and the convolution have no memory: the same with T = 1.  The norm's gradient is what a projection leaves
  over, so its errors go by the size of the vector that is projected.
* A sum over n terms: 2^-22 (16 + sqrt n) of the sum of the terms' magnitudes.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_gdn_gb300 as gdn
import mixer_reference as R
from mixer_reference import f64

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_rule_gdn_gb300 import build
    build.build()
    gdn.load()
    yield
    torch.cuda.synchronize()
    assert gdn.device_status() == 0


def close(got, ref, what, T=1, grad=False, size=0.0):
    """``ref``: the reference, or another computed tensor (then both sides may be off: twice the tolerance)."""
    sides = 1.0
    if isinstance(ref, torch.Tensor):
        ref, sides = f64(ref), 2.0
    x = f64(got)
    assert x.shape == ref.shape, (what, x.shape, ref.shape)
    assert np.array_equal(np.isnan(x), np.isnan(ref)), f"{what}: NaN elsewhere"
    ok = ~np.isnan(ref)
    x, y = x[ok], ref[ok]
    if x.size == 0:
        return
    inf = np.isinf(y)
    assert np.array_equal(x[inf], y[inf]), f"{what}: infinities"
    x, y = x[~inf], y[~inf]
    assert np.isfinite(x).all(), what
    k = 4.0 if grad else 1.0
    b = got.dtype == BF
    top = max(np.abs(y).max(initial=0.0), size)
    limit = sides * (k * 2.0 ** -22 * (8 + T) * top + (2.0 ** -8 * np.abs(y) if b else 0.0) + 2.0 ** -126)
    worst = np.abs(x - y) - limit
    assert (worst <= 0).all(), f"{what}: off by {np.abs(x - y).max():.3e} of {top:.3e}"
    norm = max(np.linalg.norm(y), size * np.sqrt(y.size))
    off = np.linalg.norm(x - y)
    allowed = (k * 2.0 ** -22 * (8 + np.sqrt(T)) + (2.0 ** -8 if b else 0.0)) * norm + 2.0 ** -126 * np.sqrt(y.size)
    assert off <= sides * allowed, f"{what}: rel-L2 {off / max(norm, 1e-300):.3e}"


def close_sum(got, ref, mags, n, what):
    x = f64(got)
    assert np.isfinite(x).all(), what
    assert (np.abs(x - ref) <= 4 * 2.0 ** -22 * (16 + np.sqrt(n)) * mags + 1e-30).all(), \
        f"{what}: off by {(np.abs(x - ref) / np.maximum(mags, 1e-30)).max():.3e} of the terms' magnitudes"


def draw(gen, *shape, dtype=F32, std=1.0):
    return (torch.randn(shape, generator=gen) * std).to(dtype).cuda()


def cut(t, layout):
    """The same values in another layout: "rows" cuts them out of a wider tensor whose gaps are NaN, "odd" out of one
    that starts one element in (so no vector access is aligned)."""
    if layout == "dense":
        return t
    pad = {"rows": 16, "odd": 3}[layout]
    off = {"rows": 8, "odd": 1}[layout]
    wide = torch.full(t.shape[:-1] + (t.shape[-1] + pad,), float("nan"), dtype=t.dtype, device=t.device)
    wide[..., off:off + t.shape[-1]] = t
    return wide[..., off:off + t.shape[-1]]


def offsets(cu):
    return None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------- gated linear recurrence

def glr_case(seed, B, T, D, dtype, gdtype, cu, act, gate, normalize, h0, layout="dense"):
    gen = torch.Generator().manual_seed(seed)
    N = B if cu is None else len(cu) - 1
    x = cut(draw(gen, B, T, D, dtype=dtype), layout)
    g = draw(gen, B, T, D)
    g = cut((g if act else -(g.exp() * 0.1)).to(gdtype), layout)
    return dict(x=x, g=g, in_gate=cut(draw(gen, B, T, D, dtype=dtype), layout) if gate else None,
                A_log=draw(gen, D, std=2.0) - 2 if act else None, dt_bias=draw(gen, D) if act else None,
                normalize=normalize, initial_state=draw(gen, N, D) if h0 else None, cu_seqlens=offsets(cu)), gen, N


def glr_check(kw, gen, N, checkpoints=True, backward=True):
    kw = dict(kw)
    x, g = kw.pop("x"), kw.pop("g")
    B, T, D = x.shape
    ref = dict(i=f64(kw["in_gate"]), A_log=f64(kw["A_log"]), dt_bias=f64(kw["dt_bias"]), normalize=kw["normalize"],
               h0=f64(kw["initial_state"]), cu=kw["cu_seqlens"])
    o_ref, hT_ref, prev = R.glr_fwd(f64(x), f64(g), **ref)
    o = torch.full((B, T, D), float("nan"), dtype=x.dtype, device="cuda")
    o, hT, ck = gdn.glr_scan_fwd(x, g, output_final_state=True, output_checkpoints=True, o=o, **kw)
    close(o, o_ref, "o", T)
    close(hT, hT_ref, "final state", T)
    starts = set() if ref["cu"] is None else set(ref["cu"].tolist())
    for k in range(ck.shape[1]):
        if k > 0 and 64 * k not in starts:
            close(ck[:, k], prev[:, 64 * k], f"checkpoint {k}", T)
    if not backward:
        return
    do, dhT = draw(gen, B, T, D, dtype=x.dtype), draw(gen, N, D)
    got = gdn.glr_scan_bwd(x, g, do, d_final_state=dhT, checkpoints=ck if checkpoints else None, **kw)
    want = R.glr_bwd(f64(x), f64(g), f64(do), f64(dhT), **ref)
    for name, t in zip(("dx", "dg", "di", "dh0", "dA_log", "ddt_bias"), got):
        given = {"di": ref["i"], "dh0": ref["h0"], "dA_log": ref["A_log"], "ddt_bias": ref["dt_bias"]}
        assert (t is None) == (name in given and given[name] is None), name
        if t is None:
            continue
        if name in ("dA_log", "ddt_bias"):
            # the terms carry the relative error of a gradient, T tokens of memory long
            close_sum(t, want[name], want["abs"][name], B * T, name)
        else:
            close(t, want[name], name, T, grad=True)


ALL = [(False, False, False), (True, True, True), (True, False, False), (False, True, True), (False, False, True),
       (True, False, True)]


@pytest.mark.parametrize("act,gate,normalize", ALL)
@pytest.mark.parametrize("dtype,gdtype", [(F32, F32), (BF, F32), (BF, BF)])
@pytest.mark.parametrize("B,T,D", [(2, 150, 136), (3, 65, 33)])
def test_recurrence(B, T, D, dtype, gdtype, act, gate, normalize):
    glr_check(*glr_case(1, B, T, D, dtype, gdtype, None, act, gate, normalize, True), checkpoints=act)


@pytest.mark.parametrize("T", [0, 1, 2, 63, 64, 65, 127, 128, 129, 511, 1000])
@pytest.mark.parametrize("h0", [False, True])
def test_recurrence_lengths(T, h0):
    glr_check(*glr_case(2, 2, T, 40, F32, F32, None, True, True, True, h0), checkpoints=h0)


@pytest.mark.parametrize("D", [1, 2, 3, 4, 31, 64, 100, 127, 128, 129, 256, 260])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_recurrence_widths(D, dtype):
    glr_check(*glr_case(3, 2, 70, D, dtype, dtype, None, True, True, True, True))


@pytest.mark.parametrize("layout", ["rows", "odd"])
@pytest.mark.parametrize("dtype,gdtype", [(F32, F32), (BF, F32), (BF, BF)])
def test_recurrence_strides(layout, dtype, gdtype):
    glr_check(*glr_case(4, 2, 200, 72, dtype, gdtype, None, True, True, True, True, layout))


@pytest.mark.parametrize("cu", [[0, 1], [0, 300], [0, 0, 300], [0, 300, 300], [0, 0, 0, 1, 1, 64, 64, 128, 129, 300, 300],
                                [0, 63, 64, 65, 130, 257, 300], list(range(0, 301)), [0, 200, 200, 200, 300]])
@pytest.mark.parametrize("dtype,gdtype", [(F32, F32), (BF, BF)])
@pytest.mark.parametrize("h0", [False, True])
def test_recurrence_packed(cu, dtype, gdtype, h0):
    glr_check(*glr_case(5, 1, cu[-1], 68, dtype, gdtype, cu, True, True, True, h0), checkpoints=h0)


def test_recurrence_many_tiles():
    """Long rows of few channels: the state crosses many tiles, with memories of up to thousands of tokens."""
    kw, gen, N = glr_case(6, 1, 20000, 5, F32, F32, [0, 7000, 7000, 13111, 20000], False, False, False, True)
    kw["g"] = -(torch.rand(1, 20000, 5, generator=gen) * torch.tensor([1e-4, 1e-3, 1e-2, 0.1, 3.0])).cuda()
    glr_check(kw, gen, N)
    kw, gen, N = glr_case(7, 2, 9000, 3, F32, F32, None, False, False, False, True)
    kw["g"] = kw["g"] * 1e-3
    glr_check(kw, gen, N, checkpoints=False)


@pytest.mark.parametrize("normalize", [False, True])
def test_recurrence_extreme_gates(normalize):
    """Decays of exactly 0 and 1, underflowing ones, and raw logits at both ends, where softplus is 0 or infinite."""
    kw, gen, N = glr_case(8, 1, 140, 12, F32, F32, None, False, True, normalize, True)
    g = kw["g"]
    g[:, 3::7] = -float("inf")
    g[:, 5::9] = 0.0
    g[:, 6::11] = -200.0
    g[:, 8::13] = -1e-30
    kw["in_gate"][:, 4::6] = float("inf")
    kw["in_gate"][:, 7::8] = -float("inf")
    glr_check(kw, gen, N)
    kw, gen, N = glr_case(9, 1, 140, 12, F32, F32, None, True, True, normalize, True)
    kw["g"][:, 3::7] = -float("inf")
    kw["g"][:, 5::9] = float("inf")
    kw["g"][:, 6::11] = -80.0
    kw["g"][:, 8::13] = 1e4
    glr_check(kw, gen, N)


def test_recurrence_keeps_nan_inside_its_sequence():
    kw, gen, N = glr_case(10, 1, 400, 36, F32, F32, [0, 100, 230, 230, 300, 400], True, True, True, True)
    kw["x"][0, 120, ::2] = float("nan")
    kw["x"][0, 310, 1] = float("inf")
    glr_check(kw, gen, N, backward=False)
    x, g = kw.pop("x"), kw.pop("g")
    do = draw(gen, 1, 400, 36)
    dx, dg, _, dh0, _, _ = gdn.glr_scan_bwd(x, g, do, **kw)
    for lo, hi, n in ((0, 100, 0), (230, 300, 3)):
        assert torch.isfinite(dx[0, lo:hi]).all() and torch.isfinite(dg[0, lo:hi]).all() and torch.isfinite(dh0[n]).all()
    do[0, 299] = float("nan")           # a gradient that is not a number stays in its sequence too
    dx = gdn.glr_scan_bwd(x, g, do, **kw)[0]
    assert torch.isfinite(dx[0, 300:]).all() and torch.isfinite(dx[0, :100]).all() and torch.isnan(dx[0, 299]).all()


def test_recurrence_packed_equals_alone():
    kw, gen, N = glr_case(11, 1, 777, 130, BF, BF, [0, 64, 200, 203, 777], True, True, True, True)
    cu = kw.pop("cu_seqlens").tolist()
    h0 = kw.pop("initial_state")
    x, g, i = kw.pop("x"), kw.pop("g"), kw.pop("in_gate")
    o, hT = gdn.glr_scan_fwd(x, g, in_gate=i, initial_state=h0, output_final_state=True, cu_seqlens=offsets(cu), **kw)
    for n in range(N):
        lo, hi = cu[n], cu[n + 1]
        on, hn = gdn.glr_scan_fwd(x[:, lo:hi], g[:, lo:hi], in_gate=i[:, lo:hi], initial_state=h0[n:n + 1],
                                  output_final_state=True, **kw)
        close(on, o[:, lo:hi], "o", hi - lo)
        close(hn, hT[n:n + 1], "state", hi - lo)


def test_recurrence_is_the_same_from_run_to_run():
    kw, gen, N = glr_case(12, 1, 6000, 200, BF, BF, [0, 2500, 6000], True, True, True, True)
    x, g = kw.pop("x"), kw.pop("g")
    do = draw(gen, 1, 6000, 200, dtype=BF)
    first = None
    for _ in range(5):
        o, hT, ck = gdn.glr_scan_fwd(x, g, output_final_state=True, output_checkpoints=True, **kw)
        got = (o, hT) + gdn.glr_scan_bwd(x, g, do, checkpoints=ck, **kw)
        got = [t for t in got if t is not None]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_recurrence_bounded_waits_give_up():
    """A tile that never hands its map on: the waits run out, the status says so, and the next call is right again."""
    kw, gen, N = glr_case(16, 1, 3000, 64, F32, F32, None, True, True, True, True)
    x, g = kw.pop("x"), kw.pop("g")
    o1, h1 = gdn.glr_scan_fwd(x, g, output_final_state=True, **kw)
    torch.cuda.synchronize()
    assert gdn.device_status() == 0
    assert gdn.load().gdn_test_inject(4) == 0
    gdn.glr_scan_fwd(x, g, **kw)
    torch.cuda.synchronize()
    assert gdn.device_status() == 4
    assert gdn.device_status() == 0
    o2, h2 = gdn.glr_scan_fwd(x, g, output_final_state=True, **kw)
    assert torch.equal(o1, o2) and torch.equal(h1, h2)


def test_recurrence_gradient_against_differences():
    """<gradient, direction> against the forward's central difference along it, in fp32 (the difference of two sums of
    magnitude L carries 2^-22 L / step; the third derivative adds step^2)."""
    kw, gen, N = glr_case(13, 2, 90, 24, F32, F32, None, True, True, True, True)
    names = ("x", "g", "in_gate", "initial_state", "A_log", "dt_bias")
    do, dhT = draw(gen, 2, 90, 24), draw(gen, 2, 24)

    def loss(p):
        p = dict(kw, **p)
        x, g = p.pop("x"), p.pop("g")
        o, hT = gdn.glr_scan_fwd(x, g, output_final_state=True, **p)
        return float((o.double() * do.double()).sum() + (hT.double() * dhT.double()).sum())
    p = dict(kw)
    x, g = p.pop("x"), p.pop("g")
    dx, dg, di, dh0, dA, ddt = gdn.glr_scan_bwd(x, g, do, d_final_state=dhT, **p)
    for name, d in zip(names, (dx, dg, di, dh0, dA, ddt)):
        v = draw(gen, *d.shape)
        v = v / v.norm()
        e = 1e-2
        diff = (loss({name: kw[name] + e * v}) - loss({name: kw[name] - e * v})) / (2 * e)
        scale = float(d.double().norm())
        assert abs(diff - float((d.double() * v.double()).sum())) <= 2e-3 * scale, name


@pytest.mark.parametrize("dtype,gdtype", [(F32, F32), (BF, F32), (BF, BF)])
@pytest.mark.parametrize("N,D,layout", [(1, 1, "dense"), (1, 2048, "dense"), (5, 130, "rows"), (7, 33, "odd"),
                                        (300, 8, "dense")])
def test_recurrence_step(N, D, layout, dtype, gdtype):
    for act, gate, normalize in ALL:
        kw, gen, _ = glr_case(14, 1, N, D, dtype, gdtype, None, act, gate, normalize, False, layout)
        x, g, i = kw["x"][0], kw["g"][0], None if kw["in_gate"] is None else kw["in_gate"][0]
        h0 = draw(gen, N, D)
        o_ref, h_ref, _ = R.glr_fwd(f64(x)[:, None], f64(g)[:, None], None if i is None else f64(i)[:, None],
                                    f64(kw["A_log"]), f64(kw["dt_bias"]), normalize, f64(h0))
        more = dict(in_gate=i, A_log=kw["A_log"], dt_bias=kw["dt_bias"], normalize=normalize)
        out = torch.full_like(h0, float("nan"))
        keep = h0.clone()
        o = gdn.glr_step(x, g, h0, state_out=out, **more)
        assert torch.equal(h0, keep)
        close(o, o_ref[:, 0], "o")
        close(out, h_ref, "state")
        o2 = gdn.glr_step(x, g, h0, **more)
        assert torch.equal(o, o2) and torch.equal(h0, out)


def test_recurrence_steps_follow_the_scan():
    kw, gen, N = glr_case(15, 3, 20, 96, BF, BF, None, True, True, True, True)
    x, g, i, h = kw.pop("x"), kw.pop("g"), kw.pop("in_gate"), kw.pop("initial_state")
    kw.pop("cu_seqlens")
    o, hT = gdn.glr_scan_fwd(x, g, in_gate=i, initial_state=h, output_final_state=True, **kw)
    state = h.clone()
    for t in range(20):
        ot = gdn.glr_step(x[:, t], g[:, t], state, in_gate=i[:, t], **kw)
        close(ot, o[:, t], f"step {t}", 20)
    close(state, hT, "state", 20)


# ----------------------------------------------------------------------------------------------- query/key head norm

def table(P, rot):
    ang = np.arange(P)[:, None] * 10000.0 ** (-np.arange(rot // 2) * 2.0 / max(rot, 1))
    return (torch.tensor(np.cos(ang), dtype=F32).cuda(), torch.tensor(np.sin(ang), dtype=F32).cuda())


def qk_check(seed, lead, Hq, Hk, d, rot, norm, dtype, weight=True, interleaved=False, positions=True, layout="dense",
             zero_rows=False):
    gen = torch.Generator().manual_seed(seed)
    if layout == "fused":
        p = draw(gen, *lead, (Hq + 2 * Hk) * d, dtype=dtype)
        q, k = p[..., :Hq * d].unflatten(-1, (Hq, d)), p[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d))
    else:
        q, k = cut(draw(gen, *lead, Hq, d, dtype=dtype), layout), cut(draw(gen, *lead, Hk, d, dtype=dtype), layout)
    if zero_rows:
        q[0, ..., 0, :] = 0
        k[-1] = 0
    kw = dict(norm=norm, eps=1e-6, interleaved=interleaved)
    if weight:
        kw.update(q_weight=draw(gen, d) + 1, k_weight=draw(gen, d) + 1)
    P, pos = 2048, None
    if rot:
        kw["cos"], kw["sin"] = table(P, rot)
        if positions:
            pos = torch.randint(0, P, lead, generator=gen).to(torch.int32).cuda()
            kw["positions"] = pos
    at = np.broadcast_to(np.arange(lead[-1]), lead) if pos is None else pos.cpu().numpy()
    cos, sin = (f64(kw["cos"])[at], f64(kw["sin"])[at]) if rot else (None, None)
    dq, dk = draw(gen, *lead, Hq, d, dtype=dtype), draw(gen, *lead, Hk, d, dtype=dtype)
    outs = [torch.full(lead + (H, d), float("nan"), dtype=dtype, device="cuda") for H in (Hq, Hk)]
    yq, yk = gdn.gdn_qk_norm_fwd(q, k, q_out=outs[0], k_out=outs[1], **kw)
    gq, gk, gwq, gwk = gdn.gdn_qk_norm_bwd(q, k, dq, dk, **kw)
    n = int(np.prod(lead))
    for name, x, w, y, dy, gx, gw in (("q", q, "q_weight", yq, dq, gq, gwq), ("k", k, "k_weight", yk, dk, gk, gwk)):
        w = f64(kw.get(w))
        close(y, R.head_norm_fwd(f64(x), w, norm == "l2", 1e-6, cos, sin, interleaved), name)
        rx, rw, mags, size = R.head_norm_bwd(f64(x), w, norm == "l2", 1e-6, cos, sin, interleaved, f64(dy))
        close(gx, rx, "d" + name, grad=True, size=size)
        assert (gw is None) == (w is None)
        if w is not None:
            close_sum(gw, rw, mags, n * x.shape[-2], "dw" + name)


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rot,interleaved", [(0, False), (128, False), (64, False), (64, True), (2, False), (126, True),
                                             (10, False)])
def test_head_norm(norm, dtype, rot, interleaved):
    qk_check(1, (2, 37), 4, 2, 128, rot, norm, dtype, interleaved=interleaved)


@pytest.mark.parametrize("d", [1, 2, 3, 7, 8, 16, 31, 32, 33, 64, 80, 96, 100, 127, 128, 160, 192, 200, 255, 256])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("interleaved", [False, True])
def test_head_norm_sizes(d, dtype, interleaved):
    qk_check(2, (3, 5), 3, 1, d, d // 2 * 2, "rms", dtype, interleaved=interleaved)
    qk_check(3, (11,), 1, 2, d, d // 4 * 2, "l2", dtype, weight=False, interleaved=interleaved)


@pytest.mark.parametrize("layout", ["fused", "rows", "odd"])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [128, 256, 100])
def test_head_norm_strides(layout, dtype, d):
    qk_check(4, (2, 9), 4, 2, d, d // 4 * 2, "rms", dtype, layout=layout, positions=False)


@pytest.mark.parametrize("lead,Hq,Hk", [((1, 1), 1, 1), ((1,), 32, 32), ((256,), 16, 2), ((3, 700), 5, 3), ((1, 2000), 1, 1),
                                        ((2, 3), 64, 8), ((0,), 2, 2), ((2, 0), 2, 2)])
def test_head_norm_counts(lead, Hq, Hk):
    if 0 in lead:
        q, k = torch.zeros(*lead, Hq, 64, device="cuda"), torch.zeros(*lead, Hk, 64, device="cuda")
        w = torch.ones(64, device="cuda")
        y, _ = gdn.gdn_qk_norm_fwd(q, k)
        assert y.shape == q.shape
        _, _, dw, _ = gdn.gdn_qk_norm_bwd(q, k, q, k, q_weight=w, k_weight=w)
        assert torch.equal(dw, torch.zeros_like(w))
        return
    qk_check(5, lead, Hq, Hk, 128, 64, "rms", BF, positions=len(lead) == 1 or lead[1] < 1000)


def test_head_norm_zero_heads_and_weights_of_one_side():
    qk_check(6, (2, 6), 3, 2, 128, 64, "rms", F32, zero_rows=True)
    qk_check(7, (2, 6), 3, 2, 60, 0, "l2", F32, zero_rows=True, weight=False)
    q, k = torch.randn(2, 5, 2, 64, device="cuda"), torch.randn(2, 5, 1, 64, device="cuda")
    w = torch.randn(64, device="cuda")
    _, y = gdn.gdn_qk_norm_fwd(q, k, k_weight=w)
    _, y1 = gdn.gdn_qk_norm_fwd(q, k)
    close(y, f64(y1) * f64(w), "k")
    _, _, dwq, dwk = gdn.gdn_qk_norm_bwd(q, k, q, k, k_weight=w)
    assert dwq is None and dwk.shape == (64,)


def test_head_norm_positions_are_clamped_into_the_table():
    q, k = torch.randn(6, 2, 64, device="cuda"), torch.randn(6, 2, 64, device="cuda")
    cos, sin = table(10, 64)
    pos = torch.tensor([-5, 0, 9, 10, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    a, _ = gdn.gdn_qk_norm_fwd(q, k, cos=cos, sin=sin, positions=pos)
    b, _ = gdn.gdn_qk_norm_fwd(q, k, cos=cos, sin=sin, positions=pos.clamp(0, 9))
    assert torch.equal(a, b)


def test_head_norm_keeps_nan_inside_its_head():
    q, k = torch.randn(3, 4, 128, device="cuda"), torch.randn(3, 2, 128, device="cuda")
    ref, _ = gdn.gdn_qk_norm_fwd(q, k)
    q[1, 2, 5] = float("nan")
    y, yk = gdn.gdn_qk_norm_fwd(q, k)
    bad = torch.isnan(y)
    assert bad[1, 2].all() and bad.sum() == 128 and torch.equal(y[~bad], ref[~bad]) and torch.isfinite(yk).all()


def test_head_norm_gradient_against_differences():
    gen = torch.Generator().manual_seed(8)
    q, k = draw(gen, 2, 7, 3, 96), draw(gen, 2, 7, 1, 96)
    cos, sin = table(7, 48)
    kw = dict(q_weight=draw(gen, 96) + 1, k_weight=draw(gen, 96) + 1, cos=cos, sin=sin, interleaved=True)
    dq, dk = draw(gen, 2, 7, 3, 96), draw(gen, 2, 7, 1, 96)

    def loss(q, k, wq, wk):
        a, b = gdn.gdn_qk_norm_fwd(q, k, **dict(kw, q_weight=wq, k_weight=wk))
        return float((a.double() * dq.double()).sum() + (b.double() * dk.double()).sum())
    args = [q, k, kw["q_weight"], kw["k_weight"]]
    for j, d in enumerate(gdn.gdn_qk_norm_bwd(q, k, dq, dk, **kw)):
        v = draw(gen, *d.shape)
        v = v / v.norm()
        up, down = list(args), list(args)
        up[j], down[j] = args[j] + 1e-2 * v, args[j] - 1e-2 * v
        diff = (loss(*up) - loss(*down)) / 2e-2
        assert abs(diff - float((d.double() * v.double()).sum())) <= 2e-3 * float(d.double().norm()), j


# ------------------------------------------------------------------------------------------------- short convolution

def conv_check(seed, B, T, D, W, dtype, cu=None, bias=True, silu=True, h0=True, layout="dense", dhT=True):
    gen = torch.Generator().manual_seed(seed)
    N = B if cu is None else len(cu) - 1
    x = cut(draw(gen, B, T, D, dtype=dtype), layout)
    w, b = draw(gen, D, W), draw(gen, D) if bias else None
    h = draw(gen, N, W - 1, D, dtype=dtype) if h0 else None
    kw = dict(bias=b, activation="silu" if silu else None, initial_state=h, cu_seqlens=offsets(cu))
    y = torch.full((B, T, D), float("nan"), dtype=dtype, device="cuda")
    y, hT = gdn.gdn_short_conv_fwd(x, w, output_final_state=True, y=y, **kw)
    y_ref, hT_ref = R.conv_fwd(f64(x), f64(w), f64(b), silu, f64(h), cu)
    close(y, y_ref, "y")
    assert np.array_equal(f64(hT), hT_ref)
    dy, g = draw(gen, B, T, D, dtype=dtype), draw(gen, N, W - 1, D, dtype=dtype) if dhT else None
    dx, dw, db, dh0 = gdn.gdn_short_conv_bwd(x, w, dy, d_final_state=g, **kw)
    want = R.conv_bwd(f64(x), f64(w), f64(dy), f64(b), silu, f64(h), f64(g), cu)
    close(dx, want["dx"], "dx", grad=True)
    close_sum(dw, want["dw"], want["abs"]["dw"], B * T, "dw")
    assert (db is None) == (b is None) and (dh0 is None) == (h is None)
    if bias:
        close_sum(db, want["db"], want["abs"]["db"], B * T, "db")
    if h0:
        close(dh0, want["dh0"], "dh0", grad=True)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("bias,silu,h0", [(True, True, True), (False, False, False), (True, False, True), (False, True, False)])
def test_convolution(W, dtype, bias, silu, h0):
    conv_check(1, 2, 100, 136, W, dtype, bias=bias, silu=silu, h0=h0, dhT=h0)


@pytest.mark.parametrize("T", [0, 1, 2, 3, 4, 5, 31, 32, 33, 64, 65, 200])
@pytest.mark.parametrize("W", [2, 4])
def test_convolution_lengths(T, W):
    conv_check(2, 2, T, 24, W, F32)
    conv_check(2, 2, T, 24, W, BF, h0=False)


@pytest.mark.parametrize("D", [1, 2, 3, 7, 8, 9, 64, 127, 250, 256, 1000])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_convolution_widths(D, dtype):
    conv_check(3, 1, 70, D, 4, dtype)


@pytest.mark.parametrize("layout", ["rows", "odd"])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_convolution_strides(layout, dtype):
    conv_check(4, 2, 90, 72, 4, dtype, layout=layout)


@pytest.mark.parametrize("cu", [[0, 1], [0, 0, 150], [0, 150, 150], [0, 1, 1, 3, 6, 64, 64, 65, 128, 150, 150, 150],
                                list(range(0, 151)), [0, 31, 62, 95, 150]])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("h0", [False, True])
def test_convolution_packed(cu, dtype, h0):
    conv_check(5, 1, cu[-1], 40, 4, dtype, cu=cu, h0=h0)
    conv_check(6, 1, cu[-1], 9, 3, dtype, cu=cu, h0=h0, silu=False)


def test_convolution_keeps_nan_inside_its_sequence():
    gen = torch.Generator().manual_seed(7)
    x, w, cu = draw(gen, 1, 90, 16), draw(gen, 16, 4), offsets([0, 30, 60, 90])
    x[0, 59] = float("nan")
    x[0, 30] = float("inf")
    y, hT = gdn.gdn_short_conv_fwd(x, w, output_final_state=True, cu_seqlens=cu)
    assert torch.isfinite(y[0, :30]).all() and torch.isfinite(y[0, 60:]).all() and torch.isnan(hT[1, 2]).all()
    dy = draw(gen, 1, 90, 16)
    dy[0, 60] = float("nan")
    dx = gdn.gdn_short_conv_bwd(x, w, dy, cu_seqlens=cu)[0]
    assert torch.isfinite(dx[0, :30]).all() and torch.isfinite(dx[0, 61:]).all() and torch.isnan(dx[0, 60]).all()


def test_convolution_saturated_silu():
    """silu and its derivative where the exponential overflows: 0 below, the input (and 1) above."""
    x = torch.tensor([[[-1e4, -200.0, -100.0, -89.0, 0.0, 89.0, 200.0, 1e4]]], device="cuda")
    w = torch.zeros(8, 2, device="cuda")
    w[:, 1] = 1
    y, _ = gdn.gdn_short_conv_fwd(x, w)
    close(y, R.conv_fwd(f64(x), f64(w))[0], "y")
    dx = gdn.gdn_short_conv_bwd(x, w, torch.ones_like(x))[0]
    close(dx, R.conv_bwd(f64(x), f64(w), np.ones((1, 1, 8)))["dx"], "dx", grad=True)


def test_convolution_gradient_against_differences():
    gen = torch.Generator().manual_seed(8)
    x, w, b, h = draw(gen, 1, 50, 20), draw(gen, 20, 4), draw(gen, 20), draw(gen, 3, 3, 20)
    cu = offsets([0, 2, 20, 50])
    dy, dhT = draw(gen, 1, 50, 20), draw(gen, 3, 3, 20)

    def loss(x, w, b, h):
        y, hT = gdn.gdn_short_conv_fwd(x, w, bias=b, initial_state=h, output_final_state=True, cu_seqlens=cu)
        return float((y.double() * dy.double()).sum() + (hT.double() * dhT.double()).sum())
    args = [x, w, b, h]
    grads = gdn.gdn_short_conv_bwd(x, w, dy, bias=b, initial_state=h, d_final_state=dhT, cu_seqlens=cu)
    for j, d in enumerate(grads):
        v = draw(gen, *d.shape)
        v = v / v.norm()
        up, down = list(args), list(args)
        up[j], down[j] = args[j] + 1e-2 * v, args[j] - 1e-2 * v
        diff = (loss(*up) - loss(*down)) / 2e-2
        assert abs(diff - float((d.double() * v.double()).sum())) <= 2e-3 * float(d.double().norm()), j


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N,D,layout", [(1, 1, "dense"), (1, 256, "dense"), (9, 130, "rows"), (5, 33, "odd"), (300, 8, "dense")])
def test_convolution_step(W, dtype, N, D, layout):
    gen = torch.Generator().manual_seed(9)
    x = cut(draw(gen, N, D, dtype=dtype), layout)
    w, b, h = draw(gen, D, W), draw(gen, D), draw(gen, N, W - 1, D, dtype=dtype)
    y_ref, h_ref = R.conv_fwd(f64(x)[:, None], f64(w), f64(b), True, f64(h))
    out, keep = torch.full_like(h, float("nan")), h.clone()
    y = gdn.gdn_short_conv_step(x, h, w, b, state_out=out)
    assert torch.equal(h, keep)
    close(y, y_ref[:, 0], "y")
    assert np.array_equal(f64(out), h_ref)
    y2 = gdn.gdn_short_conv_step(x, h, w, b)
    assert torch.equal(y, y2) and torch.equal(h, out)


# -------------------------------------------------------------------------------------------------- streams and graphs

def test_calls_on_another_stream_and_in_a_graph():
    kw, gen, N = glr_case(20, 1, 3000, 512, BF, BF, None, True, True, True, True)
    x, g = kw.pop("x"), kw.pop("g")
    do = draw(gen, 1, 3000, 512, dtype=BF)
    w = draw(gen, 512, 4)

    def chain(**s):
        y, _ = gdn.gdn_short_conv_fwd(x, w, **s)
        o, hT, ck = gdn.glr_scan_fwd(y, g, output_final_state=True, output_checkpoints=True, **kw, **s)
        grads = gdn.glr_scan_bwd(y, g, do, checkpoints=ck, **kw, **s)
        q = o.unflatten(-1, (4, 128))
        qn, kn = gdn.gdn_qk_norm_fwd(q, q, norm="l2", **s)
        dq = gdn.gdn_qk_norm_bwd(q, q, qn, kn, norm="l2", **s)
        dx = gdn.gdn_short_conv_bwd(x, w, grads[0], **s)
        return [t for t in (y, o, hT, qn, kn, *grads, *dq, *dx) if t is not None]
    want = chain()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = chain(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain()
    for t in got:
        t.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
