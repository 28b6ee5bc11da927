"""Linear attention on the tensor cores and in fp32 beside values that are not finite, where chunks follow the one that has them.

Tolerances as in test_gpu_token_mixers.py: the rows of C that are not finite are added in fp32 with P rounded to bf16, like the others.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_gdn_gb300 as gdn
import token_mixer_reference as R
from mixer_reference import f64
from test_gpu_token_mixers import BF, draw, lin_case, near

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


def limits(algo, n):
    """(of the norm, of the largest element) of an fp32 result of n terms, and the roundings to bf16 on the way of a bf16 one."""
    tensor = algo == "tcgen05"
    return 2.0 ** -22 * (8 + np.sqrt(n)) + tensor * 2.0 ** -17, 2.0 ** -22 * (8 + n) + tensor * 2.0 ** -15, 2.0 * tensor


def bad_values(x, places, d):
    """An infinity, a NaN or both signs at these tokens, in channels of every group of 16 columns; what is beside them is finite."""
    channels = [c for c in (3, 20, 40, 60, 67, 90, 110, 127) if c < d]
    for i, t in enumerate(places):
        for j, c in enumerate(channels):
            if (i + j) % 2 == 0:
                x[0, t, 0, c] = (float("inf"), float("nan"), -float("inf"))[(i + j // 2) % 3]


PLACES = [[5], [100, 300], [0, 127, 256, 383, 640], list(range(0, 700, 64))]


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("places", range(len(PLACES)))
def test_values_of_an_early_chunk_reach_all_that_see_them(algo, d, places):
    x, kw, gen, N = lin_case(20 + places, 1, 700, 1, 1, 64, d)
    v = x["v"].clone()
    bad_values(v, PLACES[places], d)
    o, hT = gdn.lin_chunk_fwd(x["q"], x["k"], v, x["g"], output_final_state=True, algo=algo, **kw)
    with np.errstate(invalid="ignore"):
        o_ref, h_ref, _ = R.lin_fwd(*(f64(t) for t in (x["q"], x["k"], v, x["g"])), 64 ** -0.5, f64(kw["initial_state"]))
    rel, el, parts = limits(algo, 700 + 64 + d)
    near(o, o_ref, "o", rel, el, parts)
    near(hT, h_ref, "state", rel, el)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("places", range(len(PLACES)))
def test_gradients_of_an_early_chunk_in_the_walk_of_the_values(algo, d, places):
    x, kw, gen, N = lin_case(30 + places, 1, 700, 1, 1, 64, d)
    do, dhT = draw(gen, 1, 700, 1, d, dtype=BF), draw(gen, N, 1, 64, d)
    do = do.clone()
    bad_values(do, [699 - t for t in PLACES[places]], d)             # (the walk goes from the last token to the first)
    _, _, dv, _, dh0 = gdn.lin_chunk_bwd(x["q"], x["k"], x["v"], x["g"], do, d_final_state=dhT, algo=algo, **kw)
    with np.errstate(invalid="ignore"):
        want = R.lin_bwd(*(f64(x[n]) for n in "qkvg"), f64(do), 64 ** -0.5, f64(kw["initial_state"]), f64(dhT))
    rel, el, parts = limits(algo, 700 + 64 + d)
    near(dv, want[2], "dv", 4 * rel, 4 * el, parts)
    near(dh0, want[4], "dh0", 4 * rel, 4 * el)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("T", [700, 4500])                           # (one walk; segments)
@pytest.mark.parametrize("which", ["q", "k", "v", "initial_state"])
def test_infinite_inputs_reach_what_the_formula_has_them_reach(algo, T, which):
    """Whatever becomes of an infinity on the way, the same results are finite as by the definition, and those are right."""
    x, kw, gen, N = lin_case(40, 1, T, 1, 1, 64, 64)
    x, kw = {n: t.clone() for n, t in x.items()}, dict(kw, initial_state=kw["initial_state"].clone())
    if which == "initial_state":
        kw[which][0, 0, 7, 50] = float("inf")
    else:
        x[which][0, 70, 0, 50] = -float("inf")
    o, hT = gdn.lin_chunk_fwd(x["q"], x["k"], x["v"], x["g"], output_final_state=True, algo=algo, **kw)
    with np.errstate(invalid="ignore"):
        o_ref, h_ref, _ = R.lin_fwd(*(f64(x[n]) for n in "qkvg"), 64 ** -0.5, f64(kw["initial_state"]))
    rel, el, parts = limits(algo, T + 128)
    near(o, o_ref, "o", rel, el, parts)
    near(hT, h_ref, "state", rel, el)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("gate", ["token", "head"])                  # (scaled values as two numbers; as three)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("which", ["q", "k"])
@pytest.mark.parametrize("T", [700, 4400])                           # (one walk; segments)
def test_gradients_beside_queries_and_keys_that_are_not_finite(algo, gate, d, which, T):
    """A query reaches the keys' and values' gradients of the tokens before it, a key the queries' behind it and its own value's."""
    x, kw, gen, N = lin_case(50 + d, 1, T, 1, 1, d, 64, gate=gate)
    x = {n: t.clone() for n, t in x.items()}
    places = [130, 300, 511]
    bad_values(x[which], [T - 1 - t for t in places] if which == "q" else places, d)
    do, dhT = draw(gen, 1, T, 1, 64, dtype=BF), draw(gen, N, 1, d, 64)
    got = gdn.lin_chunk_bwd(x["q"], x["k"], x["v"], x["g"], do, d_final_state=dhT, algo=algo, **kw)
    with np.errstate(invalid="ignore"):
        want = R.lin_bwd(*(f64(x[n]) for n in "qkvg"), f64(do), d ** -0.5, f64(kw["initial_state"]), f64(dhT))
    rel, el, parts = limits(algo, T + 64 + d)
    for name, i, p in (("dq", 0, parts), ("dk", 1, parts), ("dv", 2, parts), ("dh0", 4, 0.0)):
        near(got[i], want[i], name, 4 * rel, 4 * el, p)
