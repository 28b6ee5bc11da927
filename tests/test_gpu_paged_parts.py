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
