"""The operators around the delta rule past the sizes where their kernels change their division of work: longer runs,
rings and slots that are refilled, blocks that go round more than once, several sequences a thread.  The references and
tolerances are those of test_gpu_mixer.py.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_gdn_gb300 as gdn
import mixer_reference_flat as flat
from mixer_reference import f64
from test_gpu_mixer import close, close_sum, cut, draw, glr_case, glr_check, offsets, qk_check

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


# ------------------------------------------------------------------------------------------------- short convolution

def documents(seed, T, n):
    """Offsets of n sequences: random lengths, and some of 0 to 5 and about 64 tokens."""
    rng = np.random.default_rng(seed)
    lens = np.where(rng.random(n) < 0.4, rng.choice([0, 1, 2, 3, 4, 5, 31, 32, 33, 63, 64, 65, 128], n), 0)
    rest = lens == 0
    lens[rest] = rng.multinomial(T - lens.sum(), rng.dirichlet(np.ones(rest.sum())))
    return [0, *np.cumsum(lens).tolist()]


# runs of 64 tokens where 4864 of them and a warp of 128 channels fill the card, else of 32 where as many of those do
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("run,B,T,D,W,n,layout", [
    (64, 2, 155_681, 4, 4, 0, "dense"), (64, 1, 311_301, 3, 3, 0, "dense"), (32, 1, 155_700, 8, 2, 0, "rows"),
    (32, 3, 51_883, 1, 4, 0, "dense"), (64, 1, 311_301, 4, 4, 900, "dense"), (32, 1, 155_700, 4, 3, 900, "rows"),
    (32, 1, 155_702, 1, 2, 3000, "dense")])
def test_convolution_long_runs(run, B, T, D, W, n, layout, dtype):
    few = lambda r: B * -(-T // r) * -(-D // 128) < 152 * 32     # noqa: E731
    assert not few(run) and (run == 64 or few(64))
    gen = torch.Generator().manual_seed(run)
    cu = documents(run, T, n) if n else None
    N = n or B
    x = cut(draw(gen, B, T, D, dtype=dtype), layout)
    w, b = draw(gen, D, W), draw(gen, D)
    h, g, dy = draw(gen, N, W - 1, D, dtype=dtype), draw(gen, N, W - 1, D, dtype=dtype), draw(gen, B, T, D, dtype=dtype)
    kw = dict(bias=b, initial_state=h, cu_seqlens=offsets(cu))
    y, hT = gdn.gdn_short_conv_fwd(x, w, output_final_state=True, y=torch.full((B, T, D), float("nan"), dtype=dtype, device="cuda"), **kw)
    dx, dw, db, dh0 = gdn.gdn_short_conv_bwd(x, w, dy, d_final_state=g, **kw)
    want = flat.conv(f64(x), f64(w), f64(dy), f64(b), True, f64(h), f64(g), cu)
    close(y, want["y"], "y")
    assert np.array_equal(f64(hT), want["hT"])
    close(dx, want["dx"], "dx", grad=True)
    close(dh0, want["dh0"], "dh0", grad=True)
    close_sum(dw, want["dw"], want["abs"]["dw"], B * T, "dw")
    close_sum(db, want["db"], want["abs"]["db"], B * T, "db")


# four sequences a thread past 152 * 2048 threads; the last thread has fewer
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N,D,W", [(155_701, 8, 4), (311_299, 4, 3), (103_802, 3, 2), (311_299, 1, 4)])
def test_convolution_step_of_many_sequences(N, D, W, dtype):
    assert N * (D // 4 if D % 4 == 0 else D) > 152 * 2048 and N % 4
    gen = torch.Generator().manual_seed(N)
    x, w, b, h = draw(gen, N, D, dtype=dtype), draw(gen, D, W), draw(gen, D), draw(gen, N, W - 1, D, dtype=dtype)
    want = flat.conv(f64(x)[:, None], f64(w), None, f64(b), True, f64(h))
    out, keep = torch.full_like(h, float("nan")), h.clone()
    y = gdn.gdn_short_conv_step(x, h, w, b, state_out=out)
    assert torch.equal(h, keep)
    close(y, want["y"][:, 0], "y")
    assert np.array_equal(f64(out), want["hT"])
    y2 = gdn.gdn_short_conv_step(x, h, w, b)
    assert torch.equal(y, y2) and torch.equal(h, out)


# ----------------------------------------------------------------------------------------------- query/key head norm

# persistent blocks hold 608 * 256 / lanes shares forward and 304 * 256 / lanes backward, and refill their slots after two
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n,Hq,Hk,d,rot,interleaved", [
    (7001, 5, 3, 128, 64, False), (7001, 5, 3, 128, 128, True), (14_001, 5, 3, 64, 32, False), (7001, 2, 1, 128, 64, False),
    (7001, 3, 3, 100, 48, False), (7001, 3, 3, 100, 48, True), (7001, 4, 1, 256, 128, False), (7001, 5, 3, 128, 0, False)])
def test_head_norm_blocks_go_round(n, Hq, Hk, d, rot, interleaved, dtype):
    qk_check(21, (n,), Hq, Hk, d, rot, "rms", dtype, interleaved=interleaved)


# a warp per head: 3648 heads at once backward
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d,rot", [(33, 12), (128, 64), (250, 0)])
def test_head_norm_warps_go_round(d, rot, dtype):
    qk_check(22, (3001,), 3, 2, d, rot, "l2", dtype, layout="odd")


# ------------------------------------------------------------------------------------------- gated linear recurrence

# 304 blocks at once and places for eight tiles each: 313 tiles a row in nine columns of blocks or more
@pytest.mark.parametrize("D,dtype,packed", [(516, BF, False), (514, F32, True), (257, BF, True)])
def test_recurrence_places_go_round(D, dtype, packed):
    T = 20_011
    cu = [0, 1, 1, 700, 704, 9000, 9064, 9100, T] if packed else None
    kw, gen, N = glr_case(23, 1, T, D, dtype, dtype, cu, True, True, True, True)
    glr_check(kw, gen, N)
