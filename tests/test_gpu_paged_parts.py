"""Attention over the paged cache where a sequence's parts are joined: head sizes and counts whose products are odd.

Tolerances as in test_gpu_token_mixers.py (test_attention).
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_gdn_gb300 as gdn
import token_mixer_reference as R
from mixer_reference import f64
from test_gpu_token_mixers import BF, F32, cache_case, draw, offsets

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_rule_gdn_gb300 import build
    build.build()
    gdn.load()
    yield
    torch.cuda.synchronize()
    assert gdn.device_status() == 0


def check(q, kc, vc, table, lengths, **kw):
    d = q.shape[-1]
    o, lse = gdn.paged_attn_step(q, kc, vc, table, offsets(lengths), output_lse=True, **kw)
    o_ref, lse_ref = R.attn(f64(q), f64(kc), f64(vc), f64(table).astype(int), lengths, d ** -0.5)
    off = 2.0 ** -24 * (4 * d ** 0.5 * np.abs(f64(q)).max() * np.abs(f64(kc)).max() + 64)            # of a p, relatively
    bf = q.dtype == BF
    limit = (2 * off + (2.0 ** -17 if bf else 0)) * np.abs(f64(vc)).max() + (2.0 ** -8 if bf else 2.0 ** -22) * np.abs(o_ref)
    assert (np.abs(f64(o) - o_ref) <= limit + 1e-30).all(), np.abs(f64(o) - o_ref).max()
    fin = np.isfinite(lse_ref)
    assert np.array_equal(fin, np.isfinite(f64(lse)))
    assert (np.abs(f64(lse)[fin] - lse_ref[fin]) <= off + 2.0 ** -22 * (1 + np.abs(lse_ref[fin]))).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,Hq,Hk,d,page,max_pages,lengths", [
    (1, 1, 1, 33, 16, 24, [384]), (1, 1, 1, 1, 8, 48, [384]), (3, 1, 1, 255, 7, 55, [385, 200, 0]), (1, 3, 3, 31, 64, 11, [700]),
    (1, 5, 1, 77, 16, 56, [895])])
def test_parts_of_odd_sizes(dtype, N, Hq, Hk, d, page, max_pages, lengths):
    assert gdn.paged_attn_workspace_size(N, Hq, Hk, d, max_pages, page) % (N * Hq * (d + 2) * 4) == 0
    gen = torch.Generator().manual_seed(d)
    kc, vc, table = cache_case(gen, N, Hk, d, page, max_pages, dtype)
    check(draw(gen, N, Hq, d, dtype=dtype), kc, vc, table, lengths)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_longest_sequences(dtype):
    """Nearly 2^31 tokens: one page of 2^20 again and again, and a last one whose last hundred tokens have half of the weight.

    A lane adds up to 2^19 terms one after another in fp32, each time off by half a step of the sum: 2^-24 2^19 of it, and as much
    for the weights' sum."""
    page, d, repeats, more = 1 << 20, 8, 2046, (1 << 20) - 300
    gen = torch.Generator().manual_seed(1)
    kc, vc = draw(gen, 2, page, 1, d, dtype=dtype), draw(gen, 2, page, 1, d, dtype=dtype)
    q = draw(gen, 1, 1, d, dtype=dtype)
    tail = slice(more - 100, more)
    unit = f64(q)[0, 0] / np.linalg.norm(f64(q))
    kc[1, tail, 0] = torch.tensor(unit * (17 * d ** 0.5 / np.linalg.norm(f64(q)))).to(dtype).cuda()
    vc[1, tail] = 4
    kc[1, more:], vc[1, more:] = float("nan"), float("inf")
    table = torch.zeros(1, repeats + 1, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    length = repeats * page + more
    assert (1 << 31) - (1 << 21) < length <= (1 << 31) - 256
    o, lse = gdn.paged_attn_step(q, kc, vc, table, offsets([length]), output_lse=True)
    p = [np.exp(f64(kc)[i, :n, 0] @ f64(q)[0, 0] * d ** -0.5) for i, n in ((0, page), (1, more))]
    total = repeats * p[0].sum() + p[1].sum()
    ref = (repeats * (p[0] @ f64(vc)[0, :, 0]) + p[1] @ f64(vc)[1, :more, 0]) / total
    share = p[1][-100:].sum() / total
    assert 0.1 < share < 0.9
    assert np.abs(f64(o)[0, 0] - ref).max() <= 2.0 ** -23 * 2 ** 19 * np.abs(ref).max() + 2.0 ** -8 * np.abs(ref).max()
    assert np.abs(f64(lse)[0, 0] - np.log(total)) <= 2.0 ** -24 * 2 ** 19 + 2.0 ** -20


@pytest.mark.parametrize("dtype,layout,d,Hq,Hk", [(BF, "dense", 128, 8, 2), (BF, "together", 64, 2, 2), (BF, "dense", 256, 5, 1), (BF, "dense", 80, 20, 1),
                                                  (BF, "odd", 64, 4, 2), (F32, "dense", 128, 4, 2)])
@pytest.mark.parametrize("lengths", [[1, 17, 200], [1, 900, 3000]])
def test_infinite_values_come_out_as_infinite(dtype, layout, d, Hq, Hk, lengths):
    """On either kernel: an infinity of its sign in the channel that it is in, no number where both signs meet or one of the values
    is none, and every other channel as ever."""
    gen = torch.Generator().manual_seed(d + len(lengths))
    page, max_pages = 16, 200
    kc, vc, table = cache_case(gen, 3, Hk, d, page, max_pages, dtype, layout)
    q, inf = draw(gen, 3, Hq, d, dtype=dtype), float("inf")
    tab = f64(table).astype(int)
    plain = gdn.paged_attn_step(q, kc, vc, table, offsets(lengths))

    def put(n, t, channel, value):
        vc[tab[n, t // page], t % page, :, channel] = value

    put(0, 0, 1, inf)                                    # the only token of its sequence, so with p = 1
    put(0, 0, d - 2, -inf)
    for n in (1, 2):
        last = lengths[n] - 1
        put(n, 0, 0, inf)
        put(n, last, 3, -inf)
        put(n, last // 2, 5, inf)                        # twice the same sign
        put(n, last // 2 + 1, 5, inf)
        put(n, 2, d - 1, inf)                            # both
        put(n, last, d - 1, -inf)
        put(n, last // 3, 6, float("nan"))
    o = gdn.paged_attn_step(q, kc, vc, table, offsets(lengths))
    with np.errstate(invalid="ignore"):
        ref, _ = R.attn(f64(q), f64(kc), f64(vc), tab, lengths, d ** -0.5)
    x = f64(o)
    assert not np.isfinite(ref[1:, :, [0, 3, 5, 6, d - 1]]).any()
    assert np.array_equal(np.isnan(x), np.isnan(ref)) and np.array_equal(np.isposinf(x), np.isposinf(ref)) and np.array_equal(np.isneginf(x), np.isneginf(ref))
    # (tokens in the order that they were taken in before, and a product left out only where it was of an infinity)
    fin = torch.from_numpy(np.isfinite(ref)).cuda()
    assert torch.equal(o[fin], plain[fin])
