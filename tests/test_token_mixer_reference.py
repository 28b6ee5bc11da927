"""The 64-bit references of linear attention and the paged cache against differences and closed forms (no GPU)."""
import numpy as np
import pytest

import token_mixer_reference as R


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("cu", [None, [0, 3, 3, 7]])
def test_gradients_against_differences(cu, per_head):
    rng = np.random.default_rng(3)
    B, T, Hk, H, dk, dv = 1 if cu else 2, 7, 1, 2, 3, 2
    N = B if cu is None else len(cu) - 1
    x = dict(q=rng.normal(size=(B, T, Hk, dk)), k=rng.normal(size=(B, T, Hk, dk)), v=rng.normal(size=(B, T, H, dv)),
             g=-np.exp(rng.normal(size=H if per_head else (B, T, H))), h0=rng.normal(size=(N, H, dk, dv)))
    do, dhT = rng.normal(size=(B, T, H, dv)), rng.normal(size=(N, H, dk, dv))

    def loss(**y):
        o, hT, _ = R.lin_fwd(y["q"], y["k"], y["v"], y["g"], 0.7, y["h0"], cu)
        return (o * do).sum() + (hT * dhT).sum()

    got = dict(zip(("q", "k", "v", "g", "h0"), R.lin_bwd(x["q"], x["k"], x["v"], x["g"], do, 0.7, x["h0"], dhT, cu)))
    for name, grad in got.items():
        assert grad.shape == x[name].shape
        for at in np.ndindex(grad.shape):
            up, down = ({**x, name: x[name].copy()} for _ in range(2))
            up[name][at] += 1e-5
            down[name][at] -= 1e-5
            want = (loss(**up) - loss(**down)) / 2e-5
            # a central difference of step h is off by h^2 times the third derivative and by 2^-52 / h
            assert abs(grad[at] - want) <= 1e-7 * (1 + abs(want)), (name, at)


def test_forward_without_decay_is_the_running_sum():
    rng = np.random.default_rng(4)
    q, k, v = (rng.normal(size=(1, 9, 2, 3)) for _ in range(3))
    o, hT, _ = R.lin_fwd(q, k, v, np.zeros(2), 1.0)
    p = np.tril(np.einsum("bthd,bshd->bhts", q, k))
    assert np.allclose(o, np.einsum("bhts,bshd->bthd", p, v), rtol=0, atol=1e-13)
    assert np.allclose(hT, np.einsum("bthk,bthv->bhkv", k, v), rtol=0, atol=1e-13)


def test_a_decay_of_minus_infinity_starts_anew():
    rng = np.random.default_rng(5)
    q, k, v = (rng.normal(size=(1, 8, 1, 2)) for _ in range(3))
    g = np.full((1, 8, 1), -0.1)
    g[0, 5] = -np.inf
    o, hT, _ = R.lin_fwd(q, k, v, g, 1.0, np.ones((1, 1, 2, 2)))
    o2, hT2, _ = R.lin_fwd(q[:, 5:], k[:, 5:], v[:, 5:], g[:, 5:], 1.0)
    assert np.allclose(o[:, 5:], o2) and np.allclose(hT, hT2)


def test_attention_of_one_key_is_its_value_and_pages_that_are_none_take_no_part():
    rng = np.random.default_rng(6)
    kc, vc = (rng.normal(size=(3, 4, 1, 5)) for _ in range(2))
    q = rng.normal(size=(3, 2, 5))
    table = np.array([[2, 0], [1, -1], [7, 0]])
    o, lse = R.attn(q, kc, vc, table, [1, 8, 0], 0.5)
    assert np.allclose(o[0], vc[2, 0, 0])
    short, _ = R.attn(q[1:2], kc, vc, table[1:2], [4], 0.5)
    assert np.allclose(o[1], short[0]) and (o[2] == 0).all() and np.isneginf(lse[2]).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_turning_there_and_back(interleaved):
    rng = np.random.default_rng(7)
    x, a = rng.normal(size=(4, 2, 10)), rng.normal(size=(4, 3))
    y = R.turn(R.turn(x, np.cos(a), np.sin(a), interleaved), np.cos(a), -np.sin(a), interleaved)
    assert np.allclose(x, y, rtol=0, atol=1e-14)
