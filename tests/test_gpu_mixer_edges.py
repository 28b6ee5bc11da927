"""The operators around the delta rule at the ends of their number range, each element judged against its own size.

Tolerances, from the arithmetic (z the argument of an exponential, u = 2^-24 the unit roundoff of fp32):
* z log2 e is rounded before exp2, which moves exp(z) by |z| u of itself; the approximations of exp2, the reciprocal and
  the square root add 2^-22 each, the products and sums around them a few u.  So sigma(z), softplus(z) and what is formed
  from them are off by at most (|z| + 16) 2^-22 of themselves.
* sigma(z) below 2^-126 may count as 0: it is then off by less than 2^-126, times whatever multiplies it.
* A result in bf16 adds its unit roundoff 2^-8.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_gdn_gb300 as gdn
import mixer_reference as R
from mixer_reference import f64

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TINY = 2.0 ** -126


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_rule_gdn_gb300 import build
    build.build()
    gdn.load()
    yield
    torch.cuda.synchronize()
    assert gdn.device_status() == 0


def each(got, ref, what, rel, floor=0.0):
    """Every element within rel of its own size (and the rounding of its type), or within floor."""
    x, ref = f64(got).reshape(ref.shape), np.asarray(ref)
    limit = np.broadcast_to(np.abs(ref) * (rel + (2.0 ** -8 if got.dtype == BF else 0.0)) + floor, ref.shape)
    bad = ~(np.abs(x - ref) <= limit)
    assert not bad.any(), f"{what}: {x[bad][:4]} for {ref[bad][:4]} at {np.argwhere(bad)[:4].tolist()}"


# ------------------------------------------------------------------------------------------------- short convolution

ARGS = [-1e38, -1e36, -1e30, -1e20, -1e10, -1e4, -200.0, -100.0, -90.0, -88.0, -87.0, -60.0, -10.0, -0.5, 0.0, 0.5,
        10.0, 90.0, 1e4]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("count", [20, 19])               # four channels a thread, and one
def test_convolution_silu_of_any_argument(dtype, count):
    """silu and its derivative from the lowest finite value up, forward, backward and step."""
    x = torch.tensor(([torch.finfo(dtype).min] + ARGS)[:count], dtype=dtype).cuda()
    D = x.numel()
    w = torch.ones(D, 2, device="cuda")
    w[:, 0] = 0.5                                         # meets inputs of zero only
    p = f64(x)
    rel, one = (np.abs(p).clip(max=104) + 16) * 2.0 ** -22, np.ones((1, 1, D))
    flushed = np.abs(p).clip(max=104) * TINY              # sigma(p) < 2^-126 begins at p = -87.3, and p sigma(p) is 0 below -104
    y_ref, _ = R.conv_fwd(p[None, None], f64(w))
    y, _ = gdn.gdn_short_conv_fwd(x[None, None], w)
    each(y, y_ref, "y", rel, flushed)
    zero = torch.zeros(1, 1, D, dtype=dtype, device="cuda")
    each(gdn.gdn_short_conv_step(x[None], zero.clone(), w), y_ref[0], "step", rel, flushed)
    b = torch.zeros(D, device="cuda")
    dx, dw, db, dh0 = gdn.gdn_short_conv_bwd(x[None, None], w, torch.ones_like(x)[None, None], bias=b, initial_state=zero)
    want = R.conv_bwd(p[None, None], f64(w), one, f64(b), True, f64(zero))
    each(dx, want["dx"], "dx", rel, flushed)
    each(db, want["db"], "db", rel, flushed)
    each(dh0, want["dh0"], "dh0", rel, flushed)
    each(dw, want["dw"], "dw", np.stack([rel, rel], 1), np.stack([flushed, flushed * np.abs(p).clip(max=104)], 1))
