"""The operators around the delta rule at the ends of their number range, each element judged against its own size.

Tolerances, from the arithmetic (z the argument of an exponential, u = 2^-24 the unit roundoff of fp32):
* z log2 e is rounded before exp2, which moves exp(z) by |z| u of itself; the approximations of exp2, the reciprocal and
  the square root add 2^-22 each, the products and sums around them a few u.  So sigma(z), softplus(z) and what is formed
  from them are off by at most (|z| + 16) 2^-22 of themselves.
* sigma(z) below 2^-126 may count as 0: it is then off by less than 2^-126, times whatever multiplies it.
* A result in bf16 adds its unit roundoff 2^-8.
"""
import ctypes

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


# ------------------------------------------------------------------------------------------- gated linear recurrence

def glr_one_token(x, g, i, h0, A_log=None, dt_bias=None, normalize=False):
    """One token of one sequence, forward, step and backward with gradients of ones: (got, want), and the magnitudes
    that dg and dA_log are sums of."""
    row = lambda t: None if t is None else t[None, None]     # noqa: E731
    kw = dict(in_gate=row(i), A_log=A_log, dt_bias=dt_bias, normalize=normalize, initial_state=h0[None])
    ref = dict(i=f64(row(i)), A_log=f64(A_log), dt_bias=f64(dt_bias), normalize=normalize, h0=f64(h0[None]))
    one, x, g = torch.ones_like(row(x)), row(x), row(g)
    o, hT = gdn.glr_scan_fwd(x, g, output_final_state=True, **kw)
    state = h0[None].clone()
    gdn.glr_step(x[0], g[0], state, in_gate=None if i is None else i[None], A_log=A_log, dt_bias=dt_bias, normalize=normalize)
    got = dict(zip(("dx", "dg", "di", "dh0", "dA_log", "ddt_bias"), gdn.glr_scan_bwd(x, g, one, **kw)), hT=hT, step=state)
    want = R.glr_bwd(f64(x), f64(g), f64(one), **ref)
    want["hT"] = want["step"] = R.glr_fwd(f64(x), f64(g), **ref)[1]
    return got, want


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("count", [64, 63])
def test_recurrence_closed_input_gate(dtype, normalize, count):
    """Inputs of any finite size behind an input gate that is shut: nothing of them comes through, either way."""
    low = float(torch.finfo(dtype).min)
    gates = [-float("inf"), low, -1e30, -1e4, -200.0, -100.0, -60.0, -20.0]
    values = [low, -low, 1e30, -1e20, 1e10, -1.0, 1.0, 0.0]
    i, x = (torch.tensor(v, dtype=dtype).cuda()[:count] for v in zip(*[(a, b) for a in gates for b in values]))
    gen = torch.Generator().manual_seed(3)
    h0 = torch.randn(count, generator=gen).cuda()
    g = (-torch.rand(count, generator=gen) - 0.1).cuda()
    got, want = glr_one_token(x, g, i, h0, normalize=normalize)
    z = np.abs(f64(i)).clip(max=104)
    # what a sigma that counts as 0 leaves out; a^2 / s < 3 for these decays; a sum is off by what its larger part is
    rel, lost = (z + 16) * 2.0 ** -22, np.where(z > 87, np.abs(f64(x)) * TINY, 0)
    m, h = np.abs(f64(x)) * R.sigmoid(f64(i)), np.abs(f64(h0))
    for n in ("hT", "step"):
        each(got[n], want[n], n, 2.0 ** -20, m * rel + lost + h * 2.0 ** -20)
    each(got["dx"], want["dx"], "dx", rel, TINY)
    each(got["di"], want["di"], "di", rel, 2 * lost + TINY)
    each(got["dg"], want["dg"], "dg", 2.0 ** -20, 3 * (m * rel + lost) + h * 2.0 ** -20)


@pytest.mark.parametrize("count", [32, 31])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_recurrence_decay_next_to_one(dtype, count):
    """Log decays that are subnormal numbers: s = sqrt(1 - a^2) is about 1e-20, far inside the range of fp32, and so are
    1 / s and the gradients that have it as a factor."""
    gen = torch.Generator().manual_seed(4)
    x, i = ((torch.randn(count, generator=gen) + 0.1).to(dtype).cuda() for _ in range(2))
    h0 = torch.zeros(count, device="cuda")                # (next to a state of order one nothing of s would show)
    la = -torch.logspace(-43, -37, 32, dtype=torch.float64)[:count]
    got, want = glr_one_token(x, la.float().cuda(), i, h0, normalize=True)
    rel = (np.abs(f64(i)) + 32) * 2.0 ** -22
    for n in ("hT", "step", "dx", "di", "dg"):
        each(got[n], want[n], n, rel)
    # the same out of logits: softplus(z) = exp(z) is a normal number, times exp(A_log) it is not.  Products that are
    # subnormal are rounded in steps of 2^-149
    z = torch.linspace(-87, -80, 32)[:count].cuda()
    A = torch.full((count,), -7.0, device="cuda")
    got, want = glr_one_token(x, z, i, h0, A, torch.zeros_like(A), normalize=True)
    small = np.exp(f64(A) + f64(z))
    rel = (np.abs(f64(i)) + np.abs(f64(z)) + 32) * 2.0 ** -22 + 2 * 2.0 ** -149 / small
    for n in ("hT", "step", "dx", "di", "dA_log", "dg", "ddt_bias"):
        each(got[n], want[n], n, rel)


@pytest.mark.parametrize("count", [32, 31])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_recurrence_decay_logits_far_below_zero(dtype, count):
    """softplus(z) = exp(z) as a subnormal number, in steps of 2^-149, which the input factor (about 1e-19) still shows."""
    gen = torch.Generator().manual_seed(6)
    x, i = ((torch.randn(count, generator=gen) + 0.1).to(dtype).cuda() for _ in range(2))
    h0, z = torch.zeros(count, device="cuda"), torch.linspace(-98, -86, 32)[:count].cuda()
    A = torch.full((count,), 1.0, device="cuda")
    got, want = glr_one_token(x, z, i, h0, A, torch.zeros_like(A), normalize=True)
    small = np.exp(f64(z))
    rel = (np.abs(f64(i)) + np.abs(f64(z)) + 32) * 2.0 ** -22 + 2 * 2.0 ** -149 / small
    for n in ("hT", "step", "dx", "di", "dA_log", "dg", "ddt_bias"):
        each(got[n], want[n], n, rel)


# ----------------------------------------------------------------------------------------------- query/key head norm

@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [128, 100, 127])            # eight channels a lane, four, and a warp per head
def test_head_norm_infinities_next_to_the_rotation(dtype, d, interleaved):
    """An infinite channel that does not turn stays where it is; its neighbours are what they were."""
    gen = torch.Generator().manual_seed(5)
    q, k, dq, dk = (torch.randn(2, 5, h, d, generator=gen).to(dtype).cuda() for h in (3, 2, 3, 2))
    ang = torch.rand(5, 24, generator=gen).cuda()
    w = (torch.rand(d, generator=gen) + 0.5).cuda()
    kw = dict(cos=ang.cos(), sin=ang.sin(), interleaved=interleaved)
    bad = [50, 97]
    other = [c for c in range(d) if c not in bad]
    up = w.clone()
    up[bad] = float("inf")
    for x, y, z in zip((q, k), gdn.gdn_qk_norm_fwd(q, k, q_weight=w, k_weight=w, **kw),
                       gdn.gdn_qk_norm_fwd(q, k, q_weight=up, k_weight=up, **kw)):
        assert torch.equal(z[..., other], y[..., other])
        assert torch.equal(z[..., bad].float(), torch.copysign(torch.full_like(x[..., bad].float(), float("inf")), x[..., bad].float()))
    _, _, wq, wk = gdn.gdn_qk_norm_bwd(q, k, dq, dk, q_weight=w, k_weight=w, **kw)
    dq[0, 1, 2, bad], dk[1, 3, 0, bad] = float("inf"), float("inf")
    _, _, vq, vk = gdn.gdn_qk_norm_bwd(q, k, dq, dk, q_weight=w, k_weight=w, **kw)
    for v, was, x in ((vq, wq, q[0, 1, 2, bad]), (vk, wk, k[1, 3, 0, bad])):
        assert torch.equal(v[other], was[other])
        assert torch.equal(v[bad], torch.copysign(torch.full((2,), float("inf"), device="cuda"), x.float()))


class Pool:
    """The device's default memory pool, which cudaMallocAsync takes from: the most that was in use since reset()."""
    HIGH = 8                                              # CU_MEMPOOL_ATTR_USED_MEM_HIGH

    def __init__(self):
        self.cuda, self.pool = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p()
        assert self.cuda.cuDeviceGetDefaultMemPool(ctypes.byref(self.pool), torch.cuda.current_device()) == 0

    def reset(self):
        torch.cuda.synchronize()
        assert self.cuda.cuMemPoolSetAttribute(self.pool, self.HIGH, ctypes.byref(ctypes.c_uint64(0))) == 0
        return self.high()

    def high(self):
        torch.cuda.synchronize()
        v = ctypes.c_uint64(0)
        assert self.cuda.cuMemPoolGetAttribute(self.pool, self.HIGH, ctypes.byref(v)) == 0
        return v.value


def test_head_norm_without_weights_takes_no_workspace():
    """Only the weights' gradients need one: without weights neither the binding nor the C ABI allocates any."""
    q, k = torch.randn(2, 300, 4, 128, device="cuda"), torch.randn(2, 300, 2, 128, device="cuda")
    w = torch.ones(128, device="cuda")
    lib, pool, out = gdn.load(), Pool(), [torch.empty_like(q), torch.empty_like(k), torch.empty_like(w), torch.empty_like(w)]
    want = gdn.gdn_qk_norm_bwd(q, k, q, k, norm="l2")     # (builds what a first call builds)
    before = pool.reset()
    assert all(torch.equal(a, b) for a, b in zip(gdn.gdn_qk_norm_bwd(q, k, q, k, norm="l2")[:2], want))
    assert pool.high() == before

    def call(weight):
        p = [t.data_ptr() for t in (q, k, q, k)] + [w.data_ptr() if weight else None] * 2
        o = [t.data_ptr() for t in out[:2]] + [out[2 + i].data_ptr() if weight else None for i in (0, 1)]
        assert lib.gdn_qk_norm_bwd(*p, 1, 1e-6, None, None, 0, 0, 0, None, *o, 600, 300, 4, 2, 128, 512, 128, 256, 128, 0,
                                   None, 0, torch.cuda.current_stream().cuda_stream) == 0
        return pool.high()
    assert call(False) == before
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    assert call(True) > before                            # with weights the C ABI allocates for itself


# --------------------------------------------------------------------------------------------------------- errors

def test_a_failed_call_does_not_fail_the_next():
    """A request whose workspace no device can hold ends with the allocation's error, and the call after it is all right."""
    lib = gdn.load()
    total = torch.cuda.get_device_properties(0).total_memory
    B, T, H = 1 << 17, 1, 120
    assert gdn.workspace_size(False, B, T, H, 128, 128, 64, BF) > 1.5 * total     # (so nothing is launched)
    x, h = torch.ones(2, 64, device="cuda"), torch.zeros(2, 64, device="cuda")
    p = x.data_ptr()
    assert lib.gdn_chunk_fwd(p, p, p, p, p, 1.0, None, 0, None, None, 0, p, B, T, H, 128, 128, 64, 1, 0,
                             torch.cuda.current_stream().cuda_stream) == 3
    assert "gdn_chunk_fwd" in gdn.last_error()
    o = gdn.glr_step(x, -x, h)
    assert torch.equal(o, x) and torch.equal(h, x)
