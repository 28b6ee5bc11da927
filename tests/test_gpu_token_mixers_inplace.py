"""Buffers that a program uses twice: a state that goes in and comes out of the same place, attention whose output is its query."""
import pytest
import torch

import gated_delta_rule_gdn_gb300 as gdn
from test_gpu_token_mixers import BF, F32, cache_case, draw, lin_case, offsets

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_rule_gdn_gb300 import build
    build.build()
    gdn.load()
    yield
    torch.cuda.synchronize()
    assert gdn.device_status() == 0


@pytest.mark.parametrize("algo,dtype", [("generic", F32), ("generic", BF), ("tcgen05", BF)])
@pytest.mark.parametrize("T,cu", [(300, None), (4500, None), (4400, [0, 0, 1, 3300, 3300, 4400])])
def test_a_state_of_linear_attention_in_its_place(algo, dtype, T, cu):
    x, kw, gen, N = lin_case(60, 1, T, 1, 2, 64, 72, dtype, cu)
    o, hT = gdn.lin_chunk_fwd(x["q"], x["k"], x["v"], x["g"], output_final_state=True, algo=algo, **kw)
    state = kw["initial_state"].clone()
    o2, h2 = gdn.lin_chunk_fwd(x["q"], x["k"], x["v"], x["g"], algo=algo, **dict(kw, initial_state=state, final_state=state))
    assert h2 is state and torch.equal(o, o2) and torch.equal(hT, state)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_into_its_query(dtype):
    gen = torch.Generator().manual_seed(1)
    kc, vc, table = cache_case(gen, 3, 2, 64, 16, 40, dtype)
    q, lengths = draw(gen, 3, 40, 64, dtype=dtype), offsets([640, 20, 0])
    want = gdn.paged_attn_step(q, kc, vc, table, lengths)
    assert gdn.paged_attn_step(q, kc, vc, table, lengths, o=q) is q and torch.equal(q, want)
