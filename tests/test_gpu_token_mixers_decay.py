"""The gradient of a constant decay, a sum over all tokens in which the errors of a chunk's 128 tokens agree.

Tolerance: a chunk's part of the sum is 128 times the inner product of two states, and sums over its tokens of products of a token
with a state.  States are sums in fp32 of products whose factors are off by 2^-25 at most, so off by 2^-22 of themselves at most (each
addition of the tensor cores loses a little, in the same direction); the inner products by as much.  As a factor of the products with
tokens a state is two bf16 numbers, so each of its elements is off by 2^-17 of itself at most, with signs and tokens that are
independent: these errors add as squares, like what they are errors of.
"""
import pytest
import torch

import gated_delta_rule_gdn_gb300 as gdn
from test_gpu_token_mixers import BF, draw
from token_mixer_reference_flat import constant_decay

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_rule_gdn_gb300 import build
    build.build()
    gdn.load()
    yield
    torch.cuda.synchronize()
    assert gdn.device_status() == 0


@pytest.mark.parametrize("B,T,H,d", [(4, 4096, 16, 128), (1, 4096, 4, 128), (2, 2048, 8, 64)])      # (the second in segments)
@pytest.mark.parametrize("g", [0.0, -0.001, -0.003])
@pytest.mark.parametrize("seed", [1, 2])
def test_gradient_of_a_constant_decay(B, T, H, d, g, seed):
    gen = torch.Generator().manual_seed(seed)
    q, k, v, do = (draw(gen, B, T, H, d, dtype=BF) for _ in range(4))
    decay, dhT = torch.full((H,), g, device="cuda"), draw(gen, B, H, d, d, std=0.1)
    dg = gdn.lin_chunk_bwd(q, k, v, decay, do, d_final_state=dhT, algo="tcgen05")[3]
    want, parts = constant_decay(q, k, v, do, decay, dhT)
    limit = 2.0 ** -17 * parts[1:].square().sum((0, 1, 3)).sqrt() + 2.0 ** -22 * parts[0].abs().sum((0, 2))
    off = dg.double() - want
    assert off.norm() <= limit.norm(), f"off by {float(off.norm() / want.norm()):.2e}, limit {float(limit.norm() / want.norm()):.2e}"
