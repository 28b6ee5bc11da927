"""GPU parity of linear attention with a decay for each head, and of the paged cache's operators, against their 64-bit references.

Tolerances, from the arithmetic (u = 2^-24, e = 2^-8 the unit roundoff of bf16):
* Linear attention on the generic kernels: every result is a sum over up to T tokens and d channels whose terms have mixed signs;
  each term gathers a few roundings of u (products, decays within a chunk) and one for every chunk in its memory.  Norm:
  2^-22 (8 + sqrt(T + d)); an element: 2^-22 (8 + T + d) of the largest.  Gradients multiply up to four such factors: four times
  that.  Results in bf16 add e of the element, and of the norm.
* Linear attention on the tensor cores: tokens are bf16 and enter exactly; what is rounded on the way are the decayed scores and
  the state as an operand (once to bf16: e of each part of a bf16 result, so 2 e more, of an element's largest possible size)
  and, for what is returned in fp32, pairs of bf16 numbers (2^-17 of a term, mixed signs).
* Attention: scores are exact products summed in fp32 over d channels, so off by u d |q| |k| scale at most; p by as much
  relatively, and o by that times max |v|.
* The rotation: two products and a sum, 2 u of the pair's size, then the rounding.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_gdn_gb300 as gdn
import token_mixer_reference as R
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


def draw(gen, *shape, dtype=F32, std=1.0):
    return (torch.randn(shape, generator=gen) * std).to(dtype).cuda()


def cut(t, layout):
    """The same values in another layout: "rows" cuts token rows out of a wider tensor whose gaps are NaN, "odd" out of one that
    starts one element in, "heads" leaves gaps behind every head, "heads first" has the head dimension outside."""
    if layout == "dense":
        return t
    nan = float("nan")
    if layout == "heads":
        wide = torch.full(t.shape[:-1] + (t.shape[-1] + 8,), nan, dtype=t.dtype, device=t.device)
        wide[..., :t.shape[-1]] = t
        return wide[..., :t.shape[-1]]
    H, d = t.shape[-2:]
    pad, off = {"rows": (16, 8), "odd": (3, 1)}[layout]
    wide = torch.full(t.shape[:-2] + (H * d + pad,), nan, dtype=t.dtype, device=t.device)
    wide[..., off:off + H * d] = t.flatten(-2)
    return wide[..., off:off + H * d].unflatten(-1, (H, d))


def offsets(cu):
    return None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")


def near(got, ref, what, rel, element, parts=0.0):
    """rel: of the norm; element: of the largest; both besides the rounding of got's type.  parts: further roundings to bf16."""
    x = f64(got)
    assert x.shape == ref.shape, (what, x.shape, ref.shape)
    assert np.array_equal(np.isfinite(x), np.isfinite(ref)), f"{what}: not finite elsewhere"
    ok = np.isfinite(ref)
    x, y = x[ok], ref[ok]
    if x.size == 0:
        return
    e = 2.0 ** -8 if got.dtype == BF else 0.0
    top = np.abs(y).max()
    worst = np.abs(x - y) - (element + parts * 2.0 ** -8) * top - e * np.abs(y) - 2.0 ** -126
    assert (worst <= 0).all(), f"{what}: off by {np.abs(x - y).max():.3e} of {top:.3e}"
    off, norm = np.linalg.norm(x - y), np.linalg.norm(y)
    assert off <= (rel + e + parts * 2.0 ** -8) * norm + 1e-30, f"{what}: rel-L2 {off / max(norm, 1e-300):.3e}"


# ------------------------------------------------------------------------------------------------- linear attention

def lin_case(seed, B, T, Hk, H, dk, dv, dtype=BF, cu=None, gate="token", h0=True, layout="dense"):
    gen = torch.Generator().manual_seed(seed)
    N = B if cu is None else len(cu) - 1
    g = {"token": lambda: -torch.exp(torch.randn(B, T, H, generator=gen) - 2),
         "head": lambda: -torch.exp(torch.randn(H, generator=gen) - 3),
         "none": lambda: torch.zeros(H),
         "strong": lambda: -torch.exp(2 * torch.randn(B, T, H, generator=gen) + 1),
         "resets": lambda: torch.where(torch.rand(B, T, H, generator=gen) < 0.02, torch.tensor(-np.inf),
                                       -torch.exp(torch.randn(B, T, H, generator=gen) - 4))}[gate]().float().cuda()
    x = dict(q=cut(draw(gen, B, T, Hk, dk, dtype=dtype), layout), k=cut(draw(gen, B, T, Hk, dk, dtype=dtype), layout),
             v=cut(draw(gen, B, T, H, dv, dtype=dtype), layout), g=g)
    return x, dict(initial_state=draw(gen, N, H, dk, dv) if h0 else None, cu_seqlens=offsets(cu)), gen, N


def lin_check(x, kw, gen, N, algo, backward=True):
    q, k, v, g = x["q"], x["k"], x["v"], x["g"]
    B, T, H, dv = v.shape
    dk = q.shape[-1]
    n, scale = T + dk + dv, dk ** -0.5
    ref = [f64(t) for t in (q, k, v, g)]
    cu, h0 = kw["cu_seqlens"], f64(kw["initial_state"])
    tensor = algo == "tcgen05"
    rel, el = 2.0 ** -22 * (8 + np.sqrt(n)), 2.0 ** -22 * (8 + n)
    fine = (rel + tensor * 2.0 ** -17, el + tensor * 2.0 ** -15)
    o_ref, hT_ref, _ = R.lin_fwd(*ref, scale, h0, cu)
    o = torch.full((B, T, H, dv), float("nan"), dtype=v.dtype, device="cuda")
    _, hT = gdn.lin_chunk_fwd(q, k, v, g, o=o, output_final_state=True, algo=algo, **kw)
    near(o, o_ref, "o", rel, el, 2.0 * tensor)
    near(hT, hT_ref, "final state", *fine)
    if not backward:
        return
    do, dhT = draw(gen, B, T, H, dv, dtype=v.dtype), draw(gen, N, H, dk, dv)
    got = gdn.lin_chunk_bwd(q, k, v, g, do, d_final_state=dhT, algo=algo, **kw)
    want = R.lin_bwd(*ref, f64(do), scale, h0, f64(dhT), cu)
    for name, a, b in zip(("dq", "dk", "dv", "dg", "dh0"), got, want):
        if name == "dh0" and h0 is None:
            assert a is None
            continue
        parts = 2.0 * tensor if name in ("dq", "dk", "dv") else 0.0
        if name == "dg" and g.dim() == 1:
            # a sum over all tokens: a token's part is off by its tolerance of the largest part, and the errors of tokens may
            # agree (those of a chunk share its sums), so the sum by no more than that of the parts' magnitudes
            each = R.lin_bwd(*ref[:3], np.broadcast_to(ref[3], (B, T, H)), f64(do), scale, h0, f64(dhT), cu)[3]
            assert (np.abs(f64(a) - b) <= 4 * fine[1] * np.abs(each).sum((0, 1)) + 1e-30).all(), name
            continue
        near(a, b, name, 4 * fine[0], 4 * fine[1], parts)


GENERIC = [
    # B, T, Hk, H, dk, dv, dtype, cu, gate, layout
    (1, 1, 1, 1, 1, 1, F32, None, "token", "dense"),
    (2, 31, 2, 2, 16, 16, F32, None, "token", "dense"),
    (1, 33, 1, 3, 40, 72, BF, None, "head", "dense"),
    (2, 100, 2, 4, 33, 31, F32, None, "none", "odd"),
    (1, 77, 1, 1, 256, 256, BF, None, "token", "rows"),
    (1, 300, 2, 2, 64, 100, BF, [0, 0, 1, 33, 33, 290, 300], "token", "heads"),
    (1, 200, 1, 2, 24, 8, F32, [0, 64, 200], "resets", "dense"),
    (1, 129, 1, 1, 32, 32, F32, None, "strong", "dense"),
    (1, 2100, 1, 2, 16, 40, F32, [0, 1024, 1024, 1030, 2100], "token", "dense"),     # many chunks, and a border on one
    (2, 1025, 1, 1, 8, 8, F32, None, "head", "dense"),
    (1, 1000, 1, 2, 40, 72, F32, None, "resets", "dense"),                           # few walks and long ones: in segments
    (2, 700, 2, 4, 64, 64, BF, None, "strong", "heads"),
    (1, 1500, 1, 1, 256, 200, F32, [0, 0, 1100, 1100, 1500], "head", "rows"),
    (1, 1300, 2, 2, 20, 256, F32, [0, 1, 1300], "token", "odd"),
]


@pytest.mark.parametrize("case", range(len(GENERIC)))
@pytest.mark.parametrize("h0", [True, False])
def test_linear_attention_generic(case, h0):
    B, T, Hk, H, dk, dv, dtype, cu, gate, layout = GENERIC[case]
    x, kw, gen, N = lin_case(case, B, T, Hk, H, dk, dv, dtype, cu, gate, h0, layout)
    lin_check(x, kw, gen, N, "generic")


TENSOR = [
    # B, T, Hk, H, dk, dv, cu, gate, layout
    (1, 1, 1, 1, 128, 128, None, "token", "dense"),
    (1, 128, 1, 1, 128, 128, None, "token", "dense"),
    (2, 129, 1, 2, 128, 128, None, "head", "rows"),
    (1, 127, 1, 1, 64, 64, None, "none", "dense"),
    (2, 300, 2, 4, 64, 128, None, "token", "heads"),
    (1, 500, 2, 2, 128, 64, None, "strong", "dense"),
    (1, 257, 1, 1, 8, 8, None, "token", "dense"),
    (1, 200, 1, 3, 40, 72, None, "token", "dense"),
    (1, 400, 1, 1, 96, 104, None, "resets", "rows"),
    (1, 700, 2, 2, 128, 128, [0, 0, 1, 130, 130, 386, 640, 700], "token", "dense"),
    (1, 900, 1, 2, 32, 128, [0, 128, 256, 900], "resets", "dense"),
    (1, 2200, 1, 1, 128, 128, [0, 1024, 1024, 1030, 2200], "head", "dense"),         # many chunks, and a border on one
    (2, 1153, 1, 1, 64, 64, None, "head", "dense"),
    (1, 4500, 1, 1, 64, 72, None, "head", "dense"),                                  # few walks and long ones: in segments
    (1, 4400, 1, 2, 24, 64, [0, 1, 1100, 1100, 3300, 4400], "token", "rows"),
    (1, 5000, 1, 1, 64, 64, [0, 0, 300, 4900, 5000], "token", "dense"),
]


@pytest.mark.parametrize("case", range(len(TENSOR)))
@pytest.mark.parametrize("h0", [True, False])
def test_linear_attention_tensor_cores(case, h0):
    B, T, Hk, H, dk, dv, cu, gate, layout = TENSOR[case]
    x, kw, gen, N = lin_case(50 + case, B, T, Hk, H, dk, dv, BF, cu, gate, h0, layout)
    lin_check(x, kw, gen, N, "tcgen05")


@pytest.mark.parametrize("T", [1, 300, 4200])
def test_linear_attention_tensor_cores_with_wide_values(T):
    x, kw, gen, N = lin_case(90, 1, T, 1, 1, 64, 200, BF)
    lin_check(x, kw, gen, N, "tcgen05", backward=False)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_linear_attention_without_tokens(dtype):
    gen = torch.Generator().manual_seed(1)
    q, v, g = torch.empty(2, 0, 1, 8, dtype=dtype, device="cuda"), torch.empty(2, 0, 2, 16, dtype=dtype, device="cuda"), \
        torch.empty(2, 0, 2, device="cuda")
    h0, dhT = draw(gen, 2, 2, 8, 16), draw(gen, 2, 2, 8, 16)
    o, hT = gdn.lin_chunk_fwd(q, q, v, g, initial_state=h0, output_final_state=True)
    assert o.shape == v.shape and torch.equal(hT, h0)
    dq, dk, dv, dg, dh0 = gdn.lin_chunk_bwd(q, q, v, g, v, initial_state=h0, d_final_state=dhT)
    assert dq.shape == q.shape and dg.shape == g.shape and torch.equal(dh0, dhT)
    *_, dg, dh0 = gdn.lin_chunk_bwd(q, q, v, torch.zeros(2, device="cuda"), v, initial_state=h0)
    assert (dg == 0).all() and (dh0 == 0).all()


@pytest.mark.parametrize("N,Hk,H,dk,dv,dtype,layout", [
    (1, 1, 1, 128, 128, BF, "dense"), (3, 2, 4, 128, 128, BF, "rows"), (2, 1, 1, 1, 1, F32, "dense"),
    (5, 1, 3, 33, 31, F32, "odd"), (4, 2, 2, 256, 256, BF, "heads"), (300, 1, 2, 64, 100, BF, "dense"),
    (2, 1, 2, 100, 36, F32, "dense")])
@pytest.mark.parametrize("in_place", [True, False])
def test_linear_attention_step(N, Hk, H, dk, dv, dtype, layout, in_place):
    gen = torch.Generator().manual_seed(N)
    q, k, v = (cut(draw(gen, N, h, d, dtype=dtype), layout) for h, d in ((Hk, dk), (Hk, dk), (H, dv)))
    g, state = -torch.exp(draw(gen, N, H)), draw(gen, N, H, dk, dv)
    g[0, 0] = -np.inf
    o_ref, h_ref, _ = R.lin_fwd(*(f64(t)[:, None] for t in (q, k, v, g)), dk ** -0.5, f64(state))
    kept, out = state.clone(), None if in_place else torch.full_like(state, float("nan"))
    o = gdn.lin_recurrent_step(q, k, v, g, state, state_out=out)
    near(o, o_ref[:, 0], "o", 2.0 ** -22 * (8 + np.sqrt(dk)), 2.0 ** -22 * (8 + dk))
    near(state if in_place else out, h_ref, "state", 2.0 ** -22 * 4, 2.0 ** -22 * 4)
    if not in_place:
        assert torch.equal(state, kept)
    # a decay for each head, and the step as a forward of one token
    o = gdn.lin_recurrent_step(q, k, v, g[0].clamp(min=-50), kept.clone())
    o2, _ = gdn.lin_chunk_fwd(q[:, None], k[:, None], v[:, None], g[0].clamp(min=-50), initial_state=kept, algo="generic")
    near(o2[:, 0], f64(o), "one token", 2.0 ** -20 + 2.0 ** -8 * (dtype == BF), 2.0 ** -18 + 2.0 ** -7 * (dtype == BF))


# ------------------------------------------------------------------------------------------------------ paged cache

def cache_case(gen, N, Hk, d, page, max_pages, dtype, layout="dense", bad=False):
    n_pages = N * max_pages + 2
    shape = (n_pages, page, Hk, d)
    if layout == "dense":
        kc, vc = draw(gen, *shape, dtype=dtype), draw(gen, *shape, dtype=dtype)
    elif layout == "together":                       # both sides of a page in one allocation
        both = draw(gen, n_pages, 2, page, Hk, d, dtype=dtype)
        kc, vc = both[:, 0], both[:, 1]
    elif layout == "heads first":
        kc, vc = (draw(gen, n_pages, Hk, page, d, dtype=dtype).transpose(1, 2) for _ in range(2))
    else:                                            # "odd": no access wider than an element is aligned
        kc, vc = (draw(gen, n_pages, page, Hk, d + 3, dtype=dtype)[..., 1:d + 1] for _ in range(2))
    table = torch.randperm(n_pages, generator=gen)[:N * max_pages].view(N, max_pages).to(torch.int32)
    if bad:
        table[0, -1] = -1
        table[-1, 0] = n_pages
    return kc, vc, table.cuda()


def tables(R_, n_pos, half):
    ang = np.arange(n_pos)[:, None] * 100.0 ** (-np.arange(half) / max(half, 1))
    return (torch.tensor(f(ang), dtype=F32, device="cuda") for f in (np.cos, np.sin)) if half else (None, None)


@pytest.mark.parametrize("new", ["one", "ragged"])
@pytest.mark.parametrize("Hq,Hk,d,rot,page,dtype,layout,interleaved", [
    (4, 2, 128, 128, 16, BF, "dense", False), (2, 2, 64, 32, 5, BF, "together", True), (0, 1, 80, 0, 24, BF, "heads first", False),
    (3, 1, 33, 22, 7, F32, "odd", True), (6, 3, 36, 36, 1, F32, "dense", False), (1, 1, 256, 64, 64, BF, "odd", False),
    (2, 1, 8, 2, 3, BF, "dense", False), (8, 4, 128, 64, 64, F32, "together", True)])
def test_append(new, Hq, Hk, d, rot, page, dtype, layout, interleaved):
    gen = torch.Generator().manual_seed(d + rot)
    N, max_pages = 5, 3
    kc, vc, table = cache_case(gen, N, Hk, d, page, max_pages, dtype, layout, bad=True)
    most = page * max_pages
    counts = [1] * N if new == "one" else [min(3, most), 0, most, 1, min(2, most)]
    # a sequence with tokens before, a full one, one past its pages, one whose positions begin before 0
    lengths = [min(counts[0] + 1, most), counts[1], most, most + 1, counts[4] - 1]
    n = sum(counts) + (2 if new == "ragged" else 0)                  # two rows behind the last sequence
    cu = None if new == "one" else np.concatenate([[0], np.cumsum(counts)])
    rows = draw(gen, n, Hq + 2 * Hk, d, dtype=dtype)
    rows = cut(rows, "odd" if layout == "odd" else "rows")
    q, k, v = (rows[:, a:b] for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)))
    cos, sin = tables(R, 40, rot // 2)
    k_ref, v_ref = f64(kc), f64(vc)
    kt, qt, vt = f64(k), f64(q), f64(v)
    q_ref = np.full((n, Hq, d), np.nan)
    wrote = np.zeros(k_ref.shape[:2], dtype=bool)
    for t, pos, pg, slot in R.places(lengths, f64(table).astype(int), page, len(k_ref), n, cu):
        at = min(max(pos, 0), 39)
        c, s = (f64(x)[at:at + 1] for x in (cos, sin)) if rot else (np.zeros((1, 0)),) * 2
        if Hq:
            q_ref[t] = R.turn(qt[t:t + 1], c, s, interleaved)[0]
        if pg is not None:
            k_ref[pg, slot], v_ref[pg, slot], wrote[pg, slot] = R.turn(kt[t:t + 1], c, s, interleaved)[0], vt[t], True
    before = kc.clone(), vc.clone()
    q_out = torch.full((n, Hq, d), float("nan"), dtype=dtype, device="cuda") if Hq else None
    got = gdn.paged_append(k, v, kc, vc, table, offsets(lengths), q=q if Hq else None, cu_seqlens=offsets(cu), cos=cos, sin=sin,
                           interleaved=interleaved, q_out=q_out)
    keep = torch.from_numpy(~wrote).cuda()
    assert torch.equal(kc[keep], before[0][keep]) and torch.equal(vc[keep], before[1][keep])
    assert np.array_equal(f64(vc), v_ref)
    # (the pair's size: an element may be small beside its partner)
    near(kc, k_ref, "keys", 2.0 ** -22, 2.0 ** -22)
    assert torch.equal(kc[..., rot:], torch.from_numpy(k_ref).to(dtype).cuda()[..., rot:])
    if Hq:
        assert got is q_out
        assert np.array_equal(np.isnan(f64(got)), np.isnan(q_ref))
        near(torch.nan_to_num(got), np.nan_to_num(q_ref), "q", 2.0 ** -22, 2.0 ** -22)
    else:
        assert got is None


ATTN = [
    # N, Hq, Hk, d, page, max_pages, dtype, layout, lengths
    (3, 4, 2, 128, 16, 4, BF, "dense", [1, 0, 64]),
    (4, 8, 8, 64, 5, 30, BF, "together", [150, 16, 17, 129]),
    (2, 16, 1, 128, 64, 20, BF, "heads first", [1280, 1000]),
    (2, 40, 2, 80, 24, 12, BF, "dense", [288, 77]),                  # 20 heads of a group: more than one tile of 16
    (1, 5, 1, 256, 7, 100, BF, "dense", [700]),
    (2, 3, 1, 100, 16, 20, BF, "odd", [320, 5]),                     # no vector access: the generic kernel
    (3, 4, 2, 128, 16, 40, F32, "dense", [640, 0, 333]),
    (2, 6, 1, 33, 3, 10, F32, "together", [30, 1]),
    (2, 2, 2, 8, 1, 9, BF, "heads first", [9, 3]),
    (1, 32, 8, 128, 64, 160, BF, "dense", [10000]),                  # many parts of one sequence
    (2, 9, 3, 256, 32, 50, F32, "dense", [1600, 1]),
    (3, 4, 4, 16, 128, 3, BF, "dense", [400, -3, 384]),              # lengths past the pages, and below 0
]


@pytest.mark.parametrize("case", range(len(ATTN)))
@pytest.mark.parametrize("bad", [False, True])
def test_attention(case, bad):
    N, Hq, Hk, d, page, max_pages, dtype, layout, lengths = ATTN[case]
    gen = torch.Generator().manual_seed(100 + case)
    kc, vc, table = cache_case(gen, N, Hk, d, page, max_pages, dtype, layout, bad)
    q = cut(draw(gen, N, Hq, d, dtype=dtype), "odd" if layout == "odd" else "heads")
    # slots that hold no token: what lies there must not matter
    live = torch.zeros(kc.shape[:2], dtype=torch.bool)
    for n, length in enumerate(lengths):
        t = np.arange(min(max(length, 0), page * max_pages))
        pages = f64(table).astype(int)[n, t // page]
        ok = (pages >= 0) & (pages < len(kc))
        live[pages[ok], t[ok] % page] = True
    kc[~live.cuda()] = float("nan")
    vc[~live.cuda()] = float("inf")
    scale = 0.3 if case % 2 else None
    o_ref, lse_ref = R.attn(f64(q), f64(kc), f64(vc), f64(table).astype(int), lengths, scale or d ** -0.5)
    o = torch.full((N, Hq, d), float("nan"), dtype=dtype, device="cuda")
    got, lse = gdn.paged_attn_step(q, kc, vc, table, offsets(lengths), scale=scale, o=o, output_lse=True)
    assert got is o
    s = (scale or d ** -0.5) * d * np.nanmax(np.abs(f64(q)), initial=0) * np.nanmax(np.abs(f64(kc)), initial=0)
    off = 2.0 ** -24 * (4 * s + 64)                  # of a p, relatively
    v_top = np.abs(f64(vc)[np.isfinite(f64(vc))]).max(initial=0.0)
    x = f64(o)
    assert np.isfinite(x).all()
    limit = (2 * off + (2.0 ** -17 if dtype == BF else 0)) * v_top + (2.0 ** -8 if dtype == BF else 2.0 ** -22) * np.abs(o_ref)
    assert (np.abs(x - o_ref) <= limit + 1e-30).all(), np.abs(x - o_ref).max()
    fin = np.isfinite(lse_ref)
    assert np.array_equal(fin, np.isfinite(f64(lse))) and np.isneginf(f64(lse)[~fin]).all()
    assert (np.abs(f64(lse)[fin] - lse_ref[fin]) <= off + 2.0 ** -22 * (1 + np.abs(lse_ref[fin]))).all()
