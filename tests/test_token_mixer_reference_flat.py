"""The chunked gradient of a constant decay against the one that goes token by token.  No GPU is needed."""
import numpy as np
import torch

import token_mixer_reference as R
from token_mixer_reference_flat import constant_decay


def test_gradient_of_a_constant_decay():
    gen = torch.Generator().manual_seed(1)
    q, k, v, do = (torch.randn(2, 384, 3, 8, generator=gen, dtype=torch.float64) for _ in range(4))
    g, dhT = torch.tensor([0.0, -0.01, -2.0]), torch.randn(2, 3, 8, 8, generator=gen)
    got, parts = constant_decay(q, k, v, do, g, dhT)
    want = R.lin_bwd(*(x.double().numpy() for x in (q, k, v, g, do)), 8 ** -0.5, None, dhT.double().numpy())[3]
    assert np.allclose(got.numpy(), want, rtol=1e-11) and parts.shape == (3, 2, 3, 3)
