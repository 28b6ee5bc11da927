"""Argument checks of linear attention and the paged cache, at the C ABI and in the binding.

Every call of the first part is refused (or answered from its sizes alone) before any CUDA work: no GPU is needed.
"""
import ctypes

import pytest
import torch

import gated_delta_rule_gdn_gb300 as gdn
from gated_delta_rule_gdn_gb300 import _binding, build

FAKE = 0x10000   # an aligned, never-dereferenced address: every call below fails validation first
INVALID, UNSUPPORTED = 1, 2
GENERIC, TWO_PASS, TCGEN05 = 1, 3, 2


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gdn.load()


def _call(f, a, kw):
    a = dict(a)
    assert set(kw) <= set(a), kw
    a.update(kw)
    return f(*a.values())


SIZES = dict(B=2, T=64, Hk=2, H=4, dk=32, dv=64, qt=64, qh=32, kt=64, kh=32, vt=256, vh=64, dtype=1)
TAIL = dict(algo=0, ws=FAKE, wsb=1 << 40, stream=None)
FWD = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, per_head=0, scale=1.0, h0=FAKE, hT=FAKE, cu=None, n=0, o=FAKE, **SIZES, **TAIL)
BWD = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, per_head=0, scale=1.0, h0=FAKE, do=FAKE, dhT=FAKE, cu=None, n=0, dq=FAKE, dK=FAKE, dV=FAKE,
           dg=FAKE, dh0=FAKE, **SIZES, **TAIL)
STEP = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, per_head=0, scale=1.0, h=FAKE, h_out=FAKE, o=FAKE, N=2, Hk=2, H=4, dk=32, dv=64, qt=64, qh=32,
            kt=64, kh=32, vt=256, vh=64, dtype=1, stream=None)
COMMON = [
    (dict(Hk=0), INVALID), (dict(H=0), INVALID), (dict(H=5), INVALID), (dict(dk=0), INVALID), (dict(dv=-1), INVALID),
    (dict(dk=257, qt=1024, qh=257, kt=1024, kh=257), UNSUPPORTED), (dict(dv=300, vt=2000, vh=300), UNSUPPORTED), (dict(dtype=2), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(g=None), INVALID), (dict(o=None), INVALID),
    (dict(q=FAKE + 1), INVALID), (dict(g=FAKE + 2), INVALID), (dict(qt=31), INVALID), (dict(qh=0), INVALID), (dict(kt=-64), INVALID),
    (dict(kh=1 << 32), INVALID), (dict(vh=63), INVALID), (dict(vt=1 << 32), INVALID),
]
CHUNK = COMMON + [
    (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(h0=FAKE + 2), INVALID), (dict(cu=FAKE, n=2), INVALID),
    (dict(B=1, cu=FAKE, n=0), INVALID), (dict(B=1, cu=FAKE + 2, n=1), INVALID), (dict(B=1 << 16, T=1 << 16), UNSUPPORTED),
    (dict(B=1, cu=FAKE, n=(1 << 30)), UNSUPPORTED), (dict(algo=TWO_PASS), INVALID), (dict(algo=9), INVALID),
    (dict(T=1 << 29, H=64, Hk=64), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", CHUNK + [(dict(hT=FAKE + 1), INVALID)])
def test_linear_attention_forward(lib, kw, status):
    assert _call(lib.lin_chunk_fwd, FWD, kw) == status
    assert "lin_chunk_fwd" in _binding.last_error()


@pytest.mark.parametrize("kw,status", [c for c in CHUNK if "o" not in c[0]] + [
    (dict(do=None), INVALID), (dict(do=FAKE + 1), INVALID), (dict(dq=None), INVALID), (dict(dK=None), INVALID), (dict(dV=None), INVALID),
    (dict(dg=None), INVALID), (dict(dg=None, per_head=1, T=0), INVALID), (dict(dhT=FAKE + 1), INVALID), (dict(dh0=FAKE + 2), INVALID),
    (dict(wsb=16), INVALID), (dict(ws=FAKE + 16), INVALID)])
def test_linear_attention_backward(lib, kw, status):
    assert _call(lib.lin_chunk_bwd, BWD, kw) == status
    assert "lin_chunk_bwd" in _binding.last_error()


@pytest.mark.parametrize("kw,status", COMMON + [(dict(N=0), INVALID), (dict(h=None), INVALID), (dict(h_out=None), INVALID), (dict(h=FAKE + 1), INVALID)])
def test_linear_attention_step(lib, kw, status):
    assert _call(lib.lin_recurrent_step, STEP, kw) == status
    assert "lin_recurrent_step" in _binding.last_error()


@pytest.mark.parametrize("kw", [dict(dtype=0), dict(dk=160, qt=320, qh=160, kt=320, kh=160), dict(dv=60, vt=256), dict(qt=68), dict(vh=68, vt=272), dict(q=FAKE + 2),
                                dict(o=FAKE + 4)])
def test_the_tensor_cores_refuse_what_does_not_fit_them(lib, kw):
    assert _call(lib.lin_chunk_fwd, FWD, dict(algo=TCGEN05, **kw)) == UNSUPPORTED
    assert "tensor-core" in _binding.last_error()


def test_workspace_sizes(lib):
    size = ctypes.c_size_t(0)
    assert lib.lin_workspace_size(0, 4, 4096, 16, 16, 128, 128, 0, ctypes.byref(size)) == 0 and size.value == 0
    one = gdn.lin_workspace_size(1, 65536, 1, 1, 128, 128)
    assert one >= 2 * 8 * 128 * 64 * 4 and one % 256 == 0            # states of segments
    assert gdn.lin_workspace_size(1, 65536, 1, 1, 128, 128, n_seqs=3) >= one
    plain, grouped = (gdn.lin_workspace_size(2, 100, h, 4, 64, 32, backward=True) for h in (4, 2))
    assert grouped - plain == 2 * 100 * 4 * 64 * 4                   # value heads' parts of dq and dk
    for bad in ((0, 0, 64, 1, 1, 8, 8, 0), (1, 1, 64, 2, 3, 8, 8, 0), (1, 1, 64, 1, 1, 8, 8, -1), (1, 2, 64, 1, 1, 8, 8, 2)):
        assert lib.lin_workspace_size(*bad, ctypes.byref(size)) == INVALID
    assert lib.lin_workspace_size(0, 1, 1, 1, 1, 8, 8, 0, None) == INVALID
    assert gdn.paged_attn_workspace_size(2, 8, 2, 64, 4, 16) == 0
    assert gdn.paged_attn_workspace_size(1, 8, 2, 64, 64, 64) % ((64 + 2) * 8 * 4) == 0
    with pytest.raises(gdn.GdnError):
        gdn.paged_attn_workspace_size(1, 3, 2, 64, 1, 1)
    assert lib.paged_attn_workspace_size(1, 2, 2, 64, 1, 1, None) == INVALID


# ------------------------------------------------------------------------------------------------------ paged cache

class Side(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("page", ctypes.c_int64), ("slot", ctypes.c_int64), ("head", ctypes.c_int64)]


class Cache(ctypes.Structure):
    _fields_ = [("k", Side), ("v", Side), ("table", ctypes.c_void_p), ("lengths", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("N", ctypes.c_int), ("max_pages", ctypes.c_int), ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("H_k", ctypes.c_int), ("d", ctypes.c_int), ("dtype", ctypes.c_int)]


def cache(**kw):
    side = kw.pop("side", {})
    a = dict(data=FAKE, page=16 * 2 * 64, slot=128, head=64)
    a.update(side)
    c = dict(table=FAKE, lengths=FAKE, table_stride=8, N=3, max_pages=8, n_pages=32, page_size=16, H_k=2, d=64, dtype=1)
    c.update(kw)
    return Cache(k=Side(**dict(a, **({} if "v_only" in kw else {}))), v=Side(**a), **c)


APPEND = dict(k=FAKE, v=FAKE, q=FAKE, cache=None, cu=None, cos=FAKE, sin=FAKE, n_pos=100, rot=64, inter=0, q_out=FAKE, n=3, Hq=4, kt=128, kh=64,
              vt=128, vh=64, qt=256, qh=64, stream=None)
ATTN = dict(q=FAKE, cache=None, scale=1.0, o=FAKE, lse=FAKE, Hq=4, qt=256, qh=64, ws=FAKE, wsb=1 << 40, stream=None)
BAD_CACHE = [
    (dict(N=-1), INVALID), (dict(n_pages=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(page_size=0), INVALID), (dict(H_k=0), INVALID),
    (dict(d=0), INVALID), (dict(d=257), UNSUPPORTED), (dict(dtype=7), INVALID), (dict(H_k=3), INVALID), (dict(table=None), INVALID),
    (dict(lengths=None), INVALID), (dict(lengths=FAKE + 2), INVALID), (dict(table=FAKE + 1), INVALID), (dict(table_stride=7), INVALID),
    (dict(max_pages=1 << 28, table_stride=1 << 28), UNSUPPORTED), (dict(N=1 << 25), UNSUPPORTED), (dict(side=dict(data=None)), INVALID),
    (dict(side=dict(data=FAKE + 1)), INVALID), (dict(side=dict(page=63)), INVALID), (dict(side=dict(slot=0)), INVALID),
    (dict(side=dict(head=-64)), INVALID), (dict(side=dict(page=1 << 41)), INVALID),
]


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_caches(lib, kw, status):
    c = cache(**kw)
    assert _call(lib.paged_append, APPEND, dict(cache=ctypes.addressof(c), n=c.N if c.N > 0 else 3)) == status
    assert "paged_append" in _binding.last_error()
    assert _call(lib.paged_attn_step, ATTN, dict(cache=ctypes.addressof(c))) == status
    assert "paged_attn_step" in _binding.last_error()


@pytest.mark.parametrize("kw", [
    dict(cache=None), dict(n=-1), dict(n=4), dict(n=1 << 32), dict(rot=63), dict(rot=66), dict(rot=-2), dict(cos=None), dict(sin=None), dict(sin=FAKE + 2),
    dict(n_pos=0), dict(cu=FAKE + 1), dict(kt=63), dict(kh=0), dict(vt=1 << 32), dict(vh=-1), dict(qt=1), dict(qh=63), dict(Hq=0), dict(Hq=3),
    dict(q=FAKE + 1), dict(q_out=None), dict(q_out=FAKE + 1), dict(k=None), dict(v=None), dict(k=FAKE + 1)])
def test_append(lib, kw):
    c = cache()
    assert _call(lib.paged_append, APPEND, dict({"cache": ctypes.addressof(c)}, **kw)) == INVALID
    assert "paged_append" in _binding.last_error()


def test_append_of_tokens_without_a_sequence(lib):
    c = cache(N=0)
    assert _call(lib.paged_append, APPEND, dict(cache=ctypes.addressof(c), cu=FAKE, n=2)) == INVALID
    assert _call(lib.paged_append, APPEND, dict(cache=ctypes.addressof(c), n=0)) == 0       # nothing to do
    assert _call(lib.paged_attn_step, ATTN, dict(cache=ctypes.addressof(c))) == 0


@pytest.mark.parametrize("kw,c", [(dict(cache=None), {}), (dict(Hq=0), {}), (dict(Hq=3), {}), (dict(q=None), {}), (dict(q=FAKE + 1), {}), (dict(o=None), {}),
                                  (dict(lse=FAKE + 2), {}), (dict(qt=63), {}), (dict(qh=1 << 32), {}), (dict(wsb=1), dict(max_pages=1000, table_stride=1000)),
                                  (dict(ws=FAKE + 8), dict(max_pages=1000, table_stride=1000))])
def test_attention(lib, kw, c):
    c = cache(**c)
    assert _call(lib.paged_attn_step, ATTN, dict({"cache": ctypes.addressof(c)}, **kw)) == INVALID
    assert "paged_attn_step" in _binding.last_error()


# -------------------------------------------------------------------------------------------------------- the binding

def test_the_binding_takes_no_tensors_of_the_host():
    build.build()
    x = torch.zeros(1, 4, 2, 8)
    g = torch.zeros(1, 4, 2)
    table, n = torch.zeros(4, 1, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    for call in (lambda: gdn.lin_chunk_fwd(x, x, x, g), lambda: gdn.lin_chunk_bwd(x, x, x, g, x),
                 lambda: gdn.lin_recurrent_step(x[0], x[0], x[0], g[0], torch.zeros(4, 2, 8, 8)),
                 lambda: gdn.paged_append(x[0], x[0], x, x, table, n), lambda: gdn.paged_attn_step(x[0], x, x, table, n)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    with pytest.raises(TypeError, match="missing argument 'g'"):
        gdn.lin_chunk_fwd(x, x, x)
    with pytest.raises(TypeError, match="unexpected keyword"):
        gdn.paged_attn_step(x, x, x, x, x, causal=True)


@pytest.mark.gpu
def test_the_binding_refuses_what_does_not_go_together():
    def z(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    q, v, g, f = z(2, 8, 1, 16), z(2, 8, 2, 32), z(2, 8, 2, dtype=torch.float32), torch.float32
    for args, kw in (((q.float(), q, v, g), {}), ((q, q[:, :4], v, g), {}), ((q, q, v, g.bfloat16()), {}), ((q, q, v, g[..., :1]), {}),
                     ((q, q, v, g[0, 0, :1]), {}), ((q[0], q, v, g), {}), ((q, q, v.half(), g), {}), ((q, q, v, g), dict(algo="two_pass")),
                     ((q, q, v, g), dict(initial_state=z(2, 2, 32, 16, dtype=f))), ((q, q, v, g), dict(initial_state=z(2, 2, 16, 32))),
                     ((q, q, v, g), dict(o=z(2, 8, 2, 16))), ((q, q, v, g), dict(cu_seqlens=z(3, dtype=torch.int64))),
                     ((q.transpose(1, 2), q, v, g), {}), ((q, q, v, g), dict(workspace=z(4)))):
        with pytest.raises((ValueError, gdn.GdnError)):
            gdn.lin_chunk_fwd(*args, **kw)
    for kw in (dict(algo=3), dict(scale="x")):
        with pytest.raises(TypeError):
            gdn.lin_chunk_fwd(q, q, v, g, **kw)
    with pytest.raises(gdn.GdnError):
        gdn.lin_chunk_fwd(q, q, v, g, cu_seqlens=torch.zeros(2, dtype=torch.int32, device="cuda"))      # B = 2
    with pytest.raises(ValueError, match="d_o"):
        gdn.lin_chunk_bwd(q, q, v, g, v[:, :4])
    kc, table, n = z(4, 16, 2, 32), z(3, 2, dtype=torch.int32), z(3, dtype=torch.int32)
    k, x = z(3, 2, 32), z(3, 4, 32)
    for args in ((x, kc, kc[:2], table, n), (x, kc.float(), kc, table, n), (x, kc, kc, table[:2], n), (x, kc, kc, table.long(), n),
                 (x, kc, kc, table, n.long()), (x[:2], kc, kc, table, n), (x, kc[0], kc[0], table, n), (x[..., :16], kc, kc, table, n),
                 (x, kc.transpose(2, 3), kc, table, n), (x, kc[..., ::2], kc[..., ::2], table, n)):
        with pytest.raises((ValueError, gdn.GdnError)):
            gdn.paged_attn_step(*args)
    cos = z(10, 8, dtype=f)
    for kw in (dict(cos=cos), dict(q_out=x), dict(cos=cos, sin=cos[:5]), dict(cos=cos[0], sin=cos[0]), dict(q=x[:2]), dict(cos=z(10, 20, dtype=f), sin=z(10, 20, dtype=f)),
               dict(cu_seqlens=z(3, dtype=torch.int32)), dict(q=z(3, 4, 16))):
        with pytest.raises((ValueError, gdn.GdnError)):
            gdn.paged_append(k, k, kc, kc, table, n, **kw)
    torch.cuda.synchronize()
