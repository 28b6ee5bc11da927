"""Linear attention and the paged cache where they can go wrong: values that are not numbers, captured graphs, other streams and
workspaces, run-to-run equality, decays at their ends, long caches, and a run of all the mixers together."""
import numpy as np
import pytest
import torch

import gated_delta_rule_gdn_gb300 as gdn
import token_mixer_reference as R
from mixer_reference import f64
from test_gpu_token_mixers import BF, F32, cache_case, draw, lin_case, lin_check, near, offsets

pytestmark = pytest.mark.gpu
ALGOS = ["generic", "tcgen05"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_rule_gdn_gb300 import build
    build.build()
    gdn.load()
    yield
    torch.cuda.synchronize()
    assert gdn.device_status() == 0


def lin_all(x, kw, do, dhT, algo, **more):
    q, k, v, g = x["q"], x["k"], x["v"], x["g"]
    o, hT = gdn.lin_chunk_fwd(q, k, v, g, output_final_state=True, algo=algo, **kw, **more)
    return (o, hT) + tuple(gdn.lin_chunk_bwd(q, k, v, g, do, d_final_state=dhT, algo=algo, **kw, **more))


def same(a, b):
    return all((x is None and y is None) or torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("which,bad", [(n, float(b)) for n in "qkvg" for b in ("nan", "inf", "-inf") if (n, b) != ("g", "inf")])
def test_a_value_that_is_not_finite_reaches_no_token_before_it(algo, which, bad):
    x, kw, gen, N = lin_case(7, 1, 600, 2, 2, 64, 64, BF, [0, 300, 600])
    t = 140                                              # in the middle of a chunk of 32 and of 128, in the first sequence
    x = {n: v.clone() for n, v in x.items()}
    clean, _ = gdn.lin_chunk_fwd(x["q"], x["k"], x["v"], x["g"], algo=algo, **kw)
    if which == "g":
        x["g"][0, t, 1] = bad
    else:
        x[which][0, t, 1, 3] = bad
    o, hT = gdn.lin_chunk_fwd(x["q"], x["k"], x["v"], x["g"], output_final_state=True, algo=algo, **kw)
    assert torch.equal(o[:, :t], clean[:, :t]) and torch.equal(o[:, 300:], clean[:, 300:])
    assert torch.equal(o[..., 0, :], clean[..., 0, :]) and torch.isfinite(hT[1]).all() and torch.isfinite(hT[0, 0]).all()
    ref, h_ref, _ = R.lin_fwd(*(f64(x[n]) for n in "qkvg"), 64 ** -0.5, f64(kw["initial_state"]), kw["cu_seqlens"])
    if which == "v":                                     # the one column it is in, from its token on
        assert np.array_equal(np.isfinite(f64(o)), np.isfinite(ref)) and not np.isfinite(ref[0, t:300, 1, 3]).any()
        assert np.array_equal(np.isfinite(f64(hT)), np.isfinite(h_ref))
    elif which == "q":
        assert not torch.isfinite(o[0, t, 1]).any() and torch.equal(o[:, t + 1:], clean[:, t + 1:])
    elif which == "g" and bad == -float("inf"):
        near(o, ref, "o", 2.0 ** -8, 2.0 ** -6)
    else:
        assert not torch.isfinite(o[0, t:300, 1]).any(-1).any()


@pytest.mark.parametrize("algo", ALGOS)
def test_gradients_of_real_tokens_survive_padding_that_is_not_finite(algo):
    # keys and values of padding behind a sequence, whose outputs have no gradient
    x, kw, gen, N = lin_case(8, 2, 200, 1, 2, 32, 64, BF, h0=False)
    x = {n: v.clone() for n, v in x.items()}
    do = draw(gen, 2, 200, 2, 64, dtype=BF)
    do[:, 150:] = 0
    x["k"][:, 150:] = 0
    clean = gdn.lin_chunk_bwd(x["q"], x["k"], x["v"], x["g"], do, algo=algo)
    x["v"][:, 150:] = float("inf")
    got = gdn.lin_chunk_bwd(x["q"], x["k"], x["v"], x["g"], do, algo=algo)
    for name, a, b in zip(("dq", "dk", "dv"), got, clean):
        assert torch.equal(a[:, :150], b[:, :150]), name


@pytest.mark.parametrize("algo", ALGOS)
def test_the_same_call_gives_the_same_bits(algo):
    x, kw, gen, N = lin_case(9, 1, 1500, 2, 4, 64, 64, BF, [0, 700, 1500], gate="head")
    do, dhT = draw(gen, 1, 1500, 4, 64, dtype=BF), draw(gen, N, 4, 64, 64)
    first = lin_all(x, kw, do, dhT, algo)
    for _ in range(3):
        assert same(first, lin_all(x, kw, do, dhT, algo))


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("T", [700, 5000])
def test_another_stream_a_given_workspace_and_a_graph(algo, T):
    x, kw, gen, N = lin_case(10, 1, T, 1, 1, 32, 32, BF)
    do, dhT = draw(gen, 1, T, 1, 32, dtype=BF), draw(gen, N, 1, 32, 32)
    want = lin_all(x, kw, do, dhT, algo)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = lin_all(x, kw, do, dhT, algo, stream=stream)
    stream.synchronize()
    assert same(want, got)
    size = max(gdn.lin_workspace_size(1, T, 1, 1, 32, 32, backward=b) for b in (False, True))
    ws = torch.full((size + 256,), 255, dtype=torch.uint8, device="cuda")     # (as NaN, and with a tail that is not touched)
    got = lin_all(x, kw, do, dhT, algo, workspace=ws[:size])
    assert same(want, got) and (ws[size:] == 255).all()
    graph = torch.cuda.CUDAGraph()
    y = {n: v.clone() for n, v in x.items()}
    with torch.cuda.graph(graph):
        out = lin_all(y, kw, do, dhT, algo)
    for _ in range(2):
        for n in y:
            y[n].copy_(x[n])
        graph.replay()
        torch.cuda.synchronize()
        assert same(want, out)


def test_two_calls_at_once():
    x, kw, gen, N = lin_case(11, 2, 900, 2, 2, 64, 64, BF)
    do, dhT = draw(gen, 2, 900, 2, 64, dtype=BF), draw(gen, N, 2, 64, 64)
    want = lin_all(x, kw, do, dhT, "auto")
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [lin_all(x, kw, do, dhT, "auto", stream=s) for s in streams]
    torch.cuda.synchronize()
    assert all(same(want, g) for g in got)


@pytest.mark.parametrize("algo", ALGOS)
def test_packed_sequences_give_the_bits_of_each_alone(algo):
    cu = [0, 5, 5, 133, 400, 1100]
    x, kw, gen, N = lin_case(12, 1, 1100, 1, 2, 64, 64, BF, cu)
    o, hT = gdn.lin_chunk_fwd(x["q"], x["k"], x["v"], x["g"], output_final_state=True, algo=algo, **kw)
    for n, (lo, hi) in enumerate(zip(cu, cu[1:])):
        if lo == hi:
            assert torch.equal(hT[n], kw["initial_state"][n])
            continue
        a, b = gdn.lin_chunk_fwd(*(x[m][:, lo:hi].contiguous() for m in "qkvg"), output_final_state=True, algo=algo,
                                 initial_state=kw["initial_state"][n:n + 1].contiguous())
        assert torch.equal(a, o[:, lo:hi]) and torch.equal(b[0], hT[n])


def test_offsets_that_are_out_of_order_stay_inside():
    x, kw, gen, N = lin_case(13, 1, 500, 1, 1, 32, 32, BF, [0, 600, -3, 200, 500])
    do = draw(gen, 1, 500, 1, 32, dtype=BF)
    for algo in ALGOS:
        lin_all(x, kw, do, None, algo)
    torch.cuda.synchronize()


@pytest.mark.parametrize("scale", [0.0, -0.5, 3.0])
@pytest.mark.parametrize("algo", ALGOS)
def test_any_scale(algo, scale):
    x, kw, gen, N = lin_case(14, 1, 150, 1, 1, 32, 32, BF)
    do, dhT = draw(gen, 1, 150, 1, 32, dtype=BF), draw(gen, N, 1, 32, 32)
    a = [f64(x[n]) for n in "qkvg"]
    o_ref, h_ref, _ = R.lin_fwd(*a, scale, f64(kw["initial_state"]))
    o, hT = gdn.lin_chunk_fwd(x["q"], x["k"], x["v"], x["g"], scale=scale, output_final_state=True, algo=algo, **kw)
    near(o, o_ref, "o", 2.0 ** -7, 2.0 ** -6)
    got = gdn.lin_chunk_bwd(x["q"], x["k"], x["v"], x["g"], do, scale=scale, d_final_state=dhT, algo=algo, **kw)
    for name, p, r in zip(("dq", "dk", "dv", "dg", "dh0"), got, R.lin_bwd(*a, f64(do), scale, f64(kw["initial_state"]), f64(dhT))):
        near(p, r, name, 2.0 ** -7 if name[1:] in "qkv" else 2.0 ** -15, 2.0 ** -6 if name[1:] in "qkv" else 2.0 ** -13)


def test_tensor_cores_and_generic_kernel_agree_past_where_walks_are_divided():
    # one walk of 40 chunks (segments), and 130 sequences (more than are sorted by their lengths)
    for seed, B, T, H, cu in ((15, 1, 5200, 1, None), (16, 1, 3000, 1, np.linspace(0, 3000, 131).astype(int).tolist())):
        x, kw, gen, N = lin_case(seed, B, T, H, H, 64, 64, BF, cu)
        do, dhT = draw(gen, B, T, H, 64, dtype=BF), draw(gen, N, H, 64, 64)
        a, b = (lin_all(x, kw, do, dhT, algo) for algo in ALGOS)
        for name, p, r in zip(("o", "state", "dq", "dk", "dv", "dg", "dh0"), a, b):
            wide = p.dtype == F32
            near(p, f64(r), name, 2.0 ** -15 if wide else 2.0 ** -6, 2.0 ** -13 if wide else 2.0 ** -5)


def test_waits_that_run_out_are_reported_and_leave_the_context_usable():
    x, kw, gen, N = lin_case(17, 1, 300, 1, 1, 64, 64, BF)
    want, _ = gdn.lin_chunk_fwd(x["q"], x["k"], x["v"], x["g"], algo="tcgen05", **kw)
    lib = gdn.load()
    assert lib.gdn_test_inject(5) == 0
    gdn.lin_chunk_fwd(x["q"], x["k"], x["v"], x["g"], algo="tcgen05", **kw)
    torch.cuda.synchronize()
    assert gdn.device_status() == 4                  # GDN_ERR_TIMEOUT, and cleared
    assert gdn.device_status() == 0
    again, _ = gdn.lin_chunk_fwd(x["q"], x["k"], x["v"], x["g"], algo="tcgen05", **kw)
    assert torch.equal(want, again)


# ------------------------------------------------------------------------------------------------------ paged cache

def test_append_and_attention_in_a_graph_on_another_stream():
    gen = torch.Generator().manual_seed(1)
    N, Hq, Hk, d, page, pages = 6, 8, 2, 128, 16, 20
    kc, vc, table = cache_case(gen, N, Hk, d, page, pages, BF)
    q, k, v = (draw(gen, N, h, d, dtype=BF) for h in (Hq, Hk, Hk))
    ang = torch.rand(320, 64, generator=gen).cuda()
    lengths = offsets([1, 320, 17, 100, 0, 256])
    kw = dict(q=q, cos=ang.cos(), sin=ang.sin())

    def step(kc, vc, **more):
        qr = gdn.paged_append(k, v, kc, vc, table, lengths, **kw, **more)
        o, lse = gdn.paged_attn_step(qr, kc, vc, table, lengths, output_lse=True, **more)
        return qr, o, lse

    a = [kc.clone(), vc.clone()]
    want = step(*a)
    b = [kc.clone(), vc.clone()]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = step(*b, stream=stream)
    stream.synchronize()
    assert same(want, got) and same(a, b)
    c = [kc.clone(), vc.clone()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*c)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert same(want, out) and same(a, c)


def test_attention_of_a_given_workspace_and_without_lse():
    gen = torch.Generator().manual_seed(2)
    kc, vc, table = cache_case(gen, 1, 1, 64, 16, 200, BF)
    q, lengths = draw(gen, 1, 2, 64, dtype=BF), offsets([3000])
    want, _ = gdn.paged_attn_step(q, kc, vc, table, lengths, output_lse=True)
    size = gdn.paged_attn_workspace_size(1, 2, 1, 64, 200, 16)
    assert size > 0
    ws = torch.full((size + 256,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(gdn.paged_attn_step(q, kc, vc, table, lengths, workspace=ws[:size]), want) and (ws[size:] == 255).all()
    assert gdn.paged_attn_workspace_size(300, 8, 8, 64, 4, 16) == 0


def test_pages_past_what_32_bits_count():
    # 2^31 elements and more into the cache, on both kernels
    d, page, Hk = 128, 64, 4
    n_pages = (1 << 31) // (page * Hk * d) + 3
    kc = torch.zeros(n_pages, page, Hk, d, dtype=BF, device="cuda")
    vc = torch.zeros(n_pages, page, Hk, d, dtype=BF, device="cuda")
    gen = torch.Generator().manual_seed(3)
    k, v, q = (draw(gen, 100, h, d, dtype=BF) for h in (Hk, Hk, 2 * Hk))
    table = torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32, device="cuda")
    gdn.paged_append(k, v, kc, vc, table, offsets([100]), cu_seqlens=offsets([0, 100]))
    assert torch.equal(kc[n_pages - 1], k[:64]) and torch.equal(vc[n_pages - 2, :36], v[64:])
    o = gdn.paged_attn_step(q[:1], kc, vc, table, offsets([100]))
    ref, _ = R.attn(f64(q[:1]), f64(k)[:, None], f64(v)[:, None], np.arange(100)[None], [100], d ** -0.5)
    near(o, ref, "o", 2.0 ** -16, 2.0 ** -14)
    # (an odd head size: the generic kernel)
    o = gdn.paged_attn_step(q[:1, :, :d - 1].contiguous(), kc[..., :d - 1], vc[..., :d - 1], table, offsets([100]))
    ref, _ = R.attn(f64(q[:1, :, :d - 1]), f64(k)[:, None, :, :d - 1], f64(v)[:, None, :, :d - 1], np.arange(100)[None], [100], (d - 1) ** -0.5)
    near(o, ref, "o", 2.0 ** -16, 2.0 ** -14)


def test_scores_at_the_ends_of_the_range():
    gen = torch.Generator().manual_seed(4)
    for dtype in (BF, F32):
        kc, vc, table = cache_case(gen, 2, 1, 32, 8, 4, dtype)
        q = draw(gen, 2, 1, 32, dtype=dtype)
        big = kc * 1e4                                   # one key takes all
        o, lse = gdn.paged_attn_step(q, big, vc, table, offsets([32, 9]), output_lse=True)
        ref, lse_ref = R.attn(f64(q), f64(big), f64(vc), f64(table).astype(int), [32, 9], 32 ** -0.5)
        near(o, ref, "o", 2.0 ** -14, 2.0 ** -12)
        assert np.allclose(f64(lse), lse_ref, rtol=1e-6)
        low = torch.full_like(kc, -3e38) * q[0].sign()   # every score -inf in fp32: no weights at all
        assert (gdn.paged_attn_step(q[:1], low, vc, table[:1], offsets([32])) == 0).all()


# ------------------------------------------------------------------------------------------------- a run of them all

def test_decoding_token_by_token_continues_a_prefill():
    """A layer of each mixer: prompts go through the chunked form and the ragged append, then tokens one at a time; both have to
    give what one pass over all tokens gives."""
    gen = torch.Generator().manual_seed(5)
    N, H, Hk, d, page, lens, more = 3, 4, 2, 64, 16, [40, 1, 133], 5
    total = [n + more for n in lens]
    cu_all, cu = np.concatenate([[0], np.cumsum(total)]), np.concatenate([[0], np.cumsum(lens)])
    q, k, v = (draw(gen, 1, cu_all[-1], h, d, dtype=BF) for h in (H, Hk, H))
    kk = k[:, :, :Hk]
    qk = q[:, :, :H]
    g = -torch.exp(draw(gen, 1, cu_all[-1], H) - 2)
    prompt = torch.cat([torch.arange(cu_all[n], cu_all[n] + lens[n]) for n in range(N)]).cuda()
    kq = qk[:, :, :Hk].contiguous()                      # linear attention's queries: one a key head
    o_all, h_all = gdn.lin_chunk_fwd(kq, kk, v, g, output_final_state=True, cu_seqlens=offsets(cu_all))
    o, state = gdn.lin_chunk_fwd(kq[:, prompt], kk[:, prompt], v[:, prompt], g[:, prompt], output_final_state=True, cu_seqlens=offsets(cu))
    near(o, f64(o_all[:, prompt]), "prefill", 2.0 ** -7, 2.0 ** -6)
    # attention over the cache of the same keys and values
    ang = torch.arange(256)[:, None] * 100.0 ** (-torch.arange(d // 2) / (d // 2))
    cos, sin = ang.cos().cuda(), ang.sin().cuda()
    kc, vc, table = cache_case(gen, N, Hk, d, page, 10, BF)
    vv = v[:, :, :Hk].contiguous()
    gdn.paged_append(kk[0, prompt], vv[0, prompt], kc, vc, table, offsets(lens), cu_seqlens=offsets(cu), cos=cos, sin=sin)
    for step in range(more):
        at = torch.tensor([cu_all[n] + lens[n] + step for n in range(N)]).cuda()
        o = gdn.lin_recurrent_step(kq[0, at], kk[0, at], v[0, at], g[0, at], state)
        near(o, f64(o_all[0, at]), "decode", 2.0 ** -7, 2.0 ** -6)
        lengths = offsets([n + step + 1 for n in lens])
        qr = gdn.paged_append(kk[0, at], vv[0, at], kc, vc, table, lengths, q=q[0, at], cos=cos, sin=sin)
        o = gdn.paged_attn_step(qr, kc, vc, table, lengths)
        for n in range(N):
            here = slice(cu_all[n], cu_all[n] + lens[n] + step + 1)
            pos = np.arange(lens[n] + step + 1)
            kr = R.turn(f64(kk[0, here]), f64(cos)[pos], f64(sin)[pos], False)
            qn = R.turn(f64(q[0, at[n]])[None], f64(cos)[pos[-1:]], f64(sin)[pos[-1:]], False)
            ref, _ = R.attn(qn, kr[:, None], f64(vv[0, here])[:, None], pos[None], [len(pos)], d ** -0.5)
            # (turned queries and keys are rounded to bf16 once: scores are off by 2^-8 |q| |k| scale, values' weights by as much)
            assert np.abs(f64(o[n]) - ref[0]).max() <= 2.0 ** -5 * np.abs(f64(vv)).max()
    near(state, f64(h_all), "state", 2.0 ** -15, 2.0 ** -13)
