"""ctypes binding of the operators around the delta rule: the gated linear recurrence, the query/key head norm with
rotation, and the short causal convolution.

Argument marshalling only, as in _binding.py.  Inputs may be cut out of a wider projection (their rows must be
contiguous and evenly spaced); outputs are contiguous.  Calls run on the current stream, or on ``stream``; with
``stream`` their outputs and workspaces are allocated on it too, so that the allocator does not hand their memory to
other streams while the call runs.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from ._binding import DTYPES, _check, load

NORMS = {"rms": 0, "l2": 1}
ACTIVATIONS = {None: 0, "silu": 1}

_F32 = torch.float32


def declare(lib):
    """Argument types of these entry points (called once, when the library is loaded)."""
    vp, fp, i, i64, sz = ctypes.c_void_p, ctypes.c_float, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    szp = ctypes.POINTER(sz)
    for name, args in {
        "glr_scan_fwd": [vp] * 5 + [i, vp, vp, vp, i, vp, vp, i, i, i, i64, i64, i64, i, i, vp, sz, vp],
        "glr_scan_bwd": [vp] * 5 + [i, vp, vp, vp, vp, i, vp, vp, vp, vp, vp, vp, vp, i, i, i, i64, i64, i64, i, i,
                                    vp, sz, vp],
        "glr_workspace_size": [i, i, i, i, i, szp],
        "glr_step": [vp] * 5 + [i, vp, vp, vp, i, i, i64, i64, i64, i, i, vp],
        "gdn_qk_norm_fwd": [vp] * 4 + [i, fp, vp, vp, i, i, i, vp, vp, vp, i64, i, i, i, i, i64, i64, i64, i64, i, vp],
        "gdn_qk_norm_bwd": [vp] * 6 + [i, fp, vp, vp, i, i, i, vp, vp, vp, vp, vp, i64, i, i, i, i, i64, i64, i64,
                                       i64, i, vp, sz, vp],
        "gdn_qk_norm_workspace_size": [i64, i, i, i, szp],
        "gdn_short_conv_fwd": [vp] * 3 + [i, vp, vp, vp, i, vp, i, i, i, i, i64, i, vp],
        "gdn_short_conv_bwd": [vp] * 3 + [i, vp, vp, vp, vp, i, vp, vp, vp, vp, i, i, i, i, i64, i, vp, sz, vp],
        "gdn_short_conv_workspace_size": [i, i, i, i, szp],
        "gdn_short_conv_step": [vp] * 3 + [i, vp, vp, vp, i, i, i, i64, i, vp],
    }.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = i, args


def _on_stream(fn):
    """Give ``fn`` a ``stream`` argument: the call and its allocations go to that stream."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _stream(x: torch.Tensor) -> int:
    index = x.device.index
    if index != torch.cuda.current_device():
        raise ValueError(f"the tensors are on cuda:{index}, the current device is cuda:{torch.cuda.current_device()}")
    return torch._C._cuda_getCurrentRawStream(index)


def _dtype(t, name) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    d = DTYPES.get(t.dtype)
    if d is None:
        raise ValueError(f"{name} must be float32 or bfloat16 (got {t.dtype})")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return d


def _tensor(t, name, shape, dtype, like):
    """Data pointer of a contiguous tensor of this shape and type (None: 0)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.shape != shape or t.dtype != dtype or t.device != like.device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {like.device} (got "
                         f"{t.dtype} {tuple(t.shape)}, strides {t.stride()}, on {t.device})")
    return t.data_ptr()


def _rows(t, name, shape, dtype, like):
    """(data pointer, row stride) of a [..., D] tensor whose rows are contiguous and evenly spaced (None: 0, 0)."""
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.shape != shape or t.dtype != dtype or t.device != like.device:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)} on {like.device} (got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device})")
    D = shape[-1]
    if t.is_contiguous():
        return t.data_ptr(), D
    return t.data_ptr(), _spacing(t, name, shape[:-1], D, t.stride()[:-1], D == 1 or t.stride(-1) == 1)


def _spacing(t, name, lead, least, strides, inner_ok):
    """The one spacing of the leading dimensions ``lead`` of a strided tensor."""
    ld, rows = None, 1
    ok = inner_ok
    for n, s in zip(reversed(lead), reversed(strides)):     # innermost leading dimension first
        if n == 1:
            continue
        if ld is None:
            ld = s
        elif s != ld * rows:
            ok = False
        rows *= n
    ld = least if ld is None else ld
    if not ok or ld < least:
        raise ValueError(f"{name} must have contiguous rows, evenly spaced (shape {tuple(t.shape)}, strides "
                         f"{t.stride()})")
    return ld


def _sequences(cu_seqlens, B, like):
    if cu_seqlens is None:
        return None, 0, B
    if not isinstance(cu_seqlens, torch.Tensor):
        raise TypeError("cu_seqlens must be a torch.Tensor")
    if (cu_seqlens.dtype != torch.int32 or cu_seqlens.device != like.device or not cu_seqlens.is_contiguous()
            or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2):
        raise ValueError(f"cu_seqlens must be a contiguous int32 vector of at least 2 offsets on {like.device}")
    n = cu_seqlens.numel() - 1
    return cu_seqlens.data_ptr(), n, n


def _workspace(workspace, need, like):
    """(pointer, bytes) of the caller's workspace, or of one from torch's caching allocator."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = torch.empty(need, dtype=torch.uint8, device=like.device)
    elif (not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8 or workspace.device != like.device
          or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {like.device}")
    return workspace.data_ptr(), workspace.numel(), workspace


# ---------------------------------------------------------------------------------------------- linear recurrence

def _glr_inputs(x, g, in_gate, A_log, dt_bias):
    dt = _dtype(x, "x")
    gdt = _dtype(g, "g")
    shape, D = x.shape, x.shape[-1]
    xp, ldx = _rows(x, "x", shape, x.dtype, x)
    gp, ldg = _rows(g, "g", shape, g.dtype, x)
    ip, ldi = _rows(in_gate, "in_gate", shape, x.dtype, x)
    Ap = _tensor(A_log, "A_log", (D,), _F32, x)
    dp = _tensor(dt_bias, "dt_bias", (D,), _F32, x)
    return (xp, gp, ip, Ap, dp), (ldx, ldg, ldi, dt, gdt)


def glr_workspace_size(B: int, T: int, D: int, n_seqs: int = 0, backward: bool = False) -> int:
    """Device workspace bytes of glr_scan_fwd, or glr_scan_bwd (C ABI glr_workspace_size)."""
    out = ctypes.c_size_t(0)
    _check(load().glr_workspace_size(int(backward), B, T, D, n_seqs, ctypes.byref(out)))
    return out.value


@_on_stream
def glr_scan_fwd(x, g, in_gate=None, A_log=None, dt_bias=None, normalize=False, initial_state=None,
                 output_final_state=False, cu_seqlens=None, o=None, final_state=None, output_checkpoints=False,
                 workspace=None):
    """Gated linear recurrence h_t = a_t h_{t-1} + u_t over whole sequences (C ABI glr_scan_fwd).

    x, g and in_gate [B, T, D]: log a = g, or -exp(A_log) softplus(g + dt_bias) with A_log; u = s sigmoid(in_gate) x
    with s = sqrt(1 - a^2) under ``normalize``.  g is fp32 or x's type; states are [N, D] fp32.  Packed sequences:
    ``cu_seqlens`` (int32, B = 1).  Returns (o in x's type, final_state or None), and with ``output_checkpoints`` the
    [B, ceil(T / 64), D] fp32 states that glr_scan_bwd takes.
    """
    lib = load()
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a [B, T, D] tensor")
    B, T, D = x.shape
    ins, lds = _glr_inputs(x, g, in_gate, A_log, dt_bias)
    cup, n_seqs, N = _sequences(cu_seqlens, B, x)
    h0 = _tensor(initial_state, "initial_state", (N, D), _F32, x)
    if o is None:
        o = torch.empty((B, T, D), dtype=x.dtype, device=x.device)
    if output_final_state and final_state is None:
        final_state = torch.empty((N, D), dtype=_F32, device=x.device)
    ck = torch.empty((B, (T + 63) // 64, D), dtype=_F32, device=x.device) if output_checkpoints else None
    ws, ws_bytes, workspace = _workspace(workspace, glr_workspace_size(B, T, D, n_seqs), x)
    _check(lib.glr_scan_fwd(*ins, bool(normalize), h0, _tensor(final_state, "final_state", (N, D), _F32, x), cup, n_seqs,
                            _tensor(o, "o", x.shape, x.dtype, x), None if ck is None else ck.data_ptr(), B, T, D,
                            *lds, ws, ws_bytes, _stream(x)))
    return (o, final_state, ck) if output_checkpoints else (o, final_state)


@_on_stream
def glr_scan_bwd(x, g, d_o, in_gate=None, A_log=None, dt_bias=None, normalize=False, initial_state=None,
                 d_final_state=None, cu_seqlens=None, checkpoints=None, workspace=None):
    """Gradients of <d_o, o> + <d_final_state, final_state> through glr_scan_fwd (C ABI glr_scan_bwd).

    ``checkpoints`` are the forward's; without them they are computed again.  Returns (dx, dg, din_gate,
    d_initial_state, dA_log, ddt_bias), with None where the input is None; token gradients in their tensor's type, the
    others fp32.
    """
    lib = load()
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a [B, T, D] tensor")
    B, T, D = x.shape
    ins, lds = _glr_inputs(x, g, in_gate, A_log, dt_bias)
    dop = _tensor(d_o, "d_o", x.shape, x.dtype, x)
    if dop is None:
        raise TypeError("d_o must be a torch.Tensor")
    cup, n_seqs, N = _sequences(cu_seqlens, B, x)
    dev = x.device
    dx, dg = torch.empty_like(d_o), torch.empty((B, T, D), dtype=g.dtype, device=dev)
    di = None if in_gate is None else torch.empty_like(d_o)
    dh0 = None if initial_state is None else torch.empty((N, D), dtype=_F32, device=dev)
    dA = None if A_log is None else torch.empty(D, dtype=_F32, device=dev)
    ddt = None if dt_bias is None else torch.empty(D, dtype=_F32, device=dev)
    ws, ws_bytes, workspace = _workspace(workspace, glr_workspace_size(B, T, D, n_seqs, True), x)
    _check(lib.glr_scan_bwd(*ins, bool(normalize), _tensor(initial_state, "initial_state", (N, D), _F32, x), dop,
                            _tensor(d_final_state, "d_final_state", (N, D), _F32, x), cup, n_seqs,
                            _tensor(checkpoints, "checkpoints", (B, (T + 63) // 64, D), _F32, x), dx.data_ptr(),
                            dg.data_ptr(), *(None if t is None else t.data_ptr() for t in (di, dh0, dA, ddt)),
                            B, T, D, *lds, ws, ws_bytes, _stream(x)))
    return dx, dg, di, dh0, dA, ddt


@_on_stream
def glr_step(x, g, state, in_gate=None, A_log=None, dt_bias=None, normalize=False, state_out=None, o=None):
    """One decode token of the gated linear recurrence for N sequences (C ABI glr_step); returns o [N, D].

    ``state`` [N, D] fp32 is updated in place, or kept when ``state_out`` is given, which then takes the new state.
    """
    lib = load()
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be an [N, D] tensor")
    N, D = x.shape
    ins, lds = _glr_inputs(x, g, in_gate, A_log, dt_bias)
    sp = _tensor(state, "state", x.shape, _F32, x)
    if o is None:
        o = torch.empty((N, D), dtype=x.dtype, device=x.device)
    _check(lib.glr_step(*ins, bool(normalize), sp, sp if state_out is None else _tensor(state_out, "state_out", x.shape, _F32, x),
                        _tensor(o, "o", x.shape, x.dtype, x), N, D, *lds, _stream(x)))
    return o


# ------------------------------------------------------------------------------------------- query/key head norm

def _heads(t, name, lead, d, dtype, like):
    """(pointer, heads, token stride, head stride) of a [..., H, d] tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() < 3 or t.shape[:-2] != lead or t.shape[-1] != d or t.dtype != dtype or t.device != like.device:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(lead)} + (heads, {d}) on {like.device} (got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device})")
    H = t.shape[-2]
    if t.is_contiguous():
        return t.data_ptr(), H, H * d, d
    s = t.stride()
    hs = s[-2] if H > 1 else d
    inner = (d == 1 or s[-1] == 1) and hs >= d
    return t.data_ptr(), H, _spacing(t, name, lead, d, s[:-2], inner), hs


def _qk_args(q, k, q_weight, k_weight, norm, eps, cos, sin, positions, interleaved):
    dt = _dtype(q, "q")
    if q.dim() < 3:
        raise ValueError("q must be a [..., heads, d] tensor")
    lead, d = q.shape[:-2], q.shape[-1]
    qp, Hq, qt, qh = _heads(q, "q", lead, d, q.dtype, q)
    kp, Hk, kt, kh = _heads(k, "k", lead, d, q.dtype, q)
    if norm not in NORMS:
        raise ValueError(f"norm must be one of {sorted(NORMS)} (got {norm!r})")
    n = 1
    for v in lead:
        n *= v
    # [B, T, heads, d]: without positions a token's position is its index in T; [N, heads, d] is one row of N tokens
    T = lead[-1] or 1
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    n_pos = rot = 0
    if cos is not None:
        if not isinstance(cos, torch.Tensor) or cos.dim() != 2:
            raise ValueError("cos must be a [positions, rotary_dim / 2] tensor")
        n_pos, rot = cos.shape[0], 2 * cos.shape[1]
    shape = (n_pos, rot // 2)
    pre = (qp, kp)
    mid = (_tensor(q_weight, "q_weight", (d,), _F32, q), _tensor(k_weight, "k_weight", (d,), _F32, q), NORMS[norm],
           float(eps), _tensor(cos, "cos", shape, _F32, q), _tensor(sin, "sin", shape, _F32, q), n_pos, rot,
           bool(interleaved), _tensor(positions, "positions", lead, torch.int32, q))
    post = (n, T, Hq, Hk, d, qt, qh, kt, kh, dt)
    return pre, mid, post


@_on_stream
def gdn_qk_norm_fwd(q, k, q_weight=None, k_weight=None, norm="rms", eps=1e-6, cos=None, sin=None, positions=None,
                    interleaved=False, q_out=None, k_out=None):
    """Norm of every query and key head, with the position rotation in the same pass (C ABI gdn_qk_norm_fwd).

    q [..., H_q, d] and k [..., H_k, d] of the same leading shape ([B, T] or [N]).  ``norm`` is "rms" (mean of squares)
    or "l2" (unit length); weights [d] fp32.  ``cos``/``sin`` [positions, rotary_dim / 2] fp32 turn the first rotary_dim
    channels, pairs (m, m + rotary_dim / 2) or (2m, 2m + 1) when ``interleaved``; ``positions`` int32 of the leading
    shape, or None: the index along its last dimension.  Returns (q_out, k_out), contiguous.
    """
    lib = load()
    pre, mid, post = _qk_args(q, k, q_weight, k_weight, norm, eps, cos, sin, positions, interleaved)
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if k_out is None:
        k_out = torch.empty(k.shape, dtype=q.dtype, device=q.device)
    _check(lib.gdn_qk_norm_fwd(*pre, *mid, _tensor(q_out, "q_out", q.shape, q.dtype, q),
                               _tensor(k_out, "k_out", k.shape, q.dtype, q), *post, _stream(q)))
    return q_out, k_out


@_on_stream
def gdn_qk_norm_bwd(q, k, d_q_out, d_k_out, q_weight=None, k_weight=None, norm="rms", eps=1e-6, cos=None, sin=None,
                    positions=None, interleaved=False, workspace=None):
    """Gradients through gdn_qk_norm_fwd (C ABI gdn_qk_norm_bwd): (dq, dk, dq_weight or None, dk_weight or None).

    d_q_out and d_k_out are contiguous, in q's type, as are dq and dk; the weights' gradients are fp32.
    """
    lib = load()
    pre, mid, post = _qk_args(q, k, q_weight, k_weight, norm, eps, cos, sin, positions, interleaved)
    dqp = _tensor(d_q_out, "d_q_out", q.shape, q.dtype, q)
    dkp = _tensor(d_k_out, "d_k_out", k.shape, q.dtype, q)
    if dqp is None or dkp is None:
        raise TypeError("d_q_out and d_k_out must be torch.Tensors")
    dq, dk = torch.empty_like(d_q_out), torch.empty_like(d_k_out)
    d = q.shape[-1]
    dwq = None if q_weight is None else torch.empty(d, dtype=_F32, device=q.device)
    dwk = None if k_weight is None else torch.empty(d, dtype=_F32, device=q.device)
    ws, ws_bytes, workspace = _workspace(workspace, qk_norm_workspace_size(post[0], post[2], post[3], d), q)
    _check(lib.gdn_qk_norm_bwd(*pre, dqp, dkp, *mid, dq.data_ptr(), dk.data_ptr(),
                               None if dwq is None else dwq.data_ptr(), None if dwk is None else dwk.data_ptr(),
                               *post, ws, ws_bytes, _stream(q)))
    return dq, dk, dwq, dwk


def qk_norm_workspace_size(n_tokens: int, H_q: int, H_k: int, d: int) -> int:
    """Device workspace bytes of gdn_qk_norm_bwd (C ABI gdn_qk_norm_workspace_size)."""
    out = ctypes.c_size_t(0)
    _check(load().gdn_qk_norm_workspace_size(n_tokens, H_q, H_k, d, ctypes.byref(out)))
    return out.value


# -------------------------------------------------------------------------------------------- short convolution

def _conv_params(x, weight, bias, activation):
    dt = _dtype(x, "x")
    D = x.shape[-1]
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a [D, W] tensor")
    W = weight.shape[1]
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be None or 'silu' (got {activation!r})")
    return dt, W, (_tensor(weight, "weight", (D, W), _F32, x), _tensor(bias, "bias", (D,), _F32, x),
                   ACTIVATIONS[activation])


@_on_stream
def gdn_short_conv_fwd(x, weight, bias=None, activation="silu", initial_state=None, output_final_state=False,
                       cu_seqlens=None, y=None, final_state=None):
    """Causal depthwise convolution of the last W tokens, with its activation (C ABI gdn_short_conv_fwd).

    x [B, T, D]; weight [D, W] (W = 2, 3, 4) and bias [D] fp32, the last tap on the current token; ``activation``
    "silu" or None.  States [N, W - 1, D] in x's type are the last W - 1 inputs, oldest first.  Returns (y,
    final_state or None).
    """
    lib = load()
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a [B, T, D] tensor")
    B, T, D = x.shape
    dt, W, params = _conv_params(x, weight, bias, activation)
    xp, ldx = _rows(x, "x", x.shape, x.dtype, x)
    cup, n_seqs, N = _sequences(cu_seqlens, B, x)
    if y is None:
        y = torch.empty((B, T, D), dtype=x.dtype, device=x.device)
    if output_final_state and final_state is None:
        final_state = torch.empty((N, W - 1, D), dtype=x.dtype, device=x.device)
    shape = (N, W - 1, D)
    _check(lib.gdn_short_conv_fwd(xp, *params, _tensor(initial_state, "initial_state", shape, x.dtype, x),
                                  _tensor(final_state, "final_state", shape, x.dtype, x), cup, n_seqs,
                                  _tensor(y, "y", x.shape, x.dtype, x), B, T, D, W, ldx, dt, _stream(x)))
    return y, final_state


def short_conv_workspace_size(B: int, T: int, D: int, W: int) -> int:
    """Device workspace bytes of gdn_short_conv_bwd (C ABI gdn_short_conv_workspace_size)."""
    out = ctypes.c_size_t(0)
    _check(load().gdn_short_conv_workspace_size(B, T, D, W, ctypes.byref(out)))
    return out.value


@_on_stream
def gdn_short_conv_bwd(x, weight, d_y, bias=None, activation="silu", initial_state=None, d_final_state=None,
                       cu_seqlens=None, workspace=None):
    """Gradients of <d_y, y> + <d_final_state, final_state> through gdn_short_conv_fwd (C ABI gdn_short_conv_bwd).

    Returns (dx, dweight, dbias, d_initial_state), the last two None where their input is None; dx and
    d_initial_state in x's type, the others fp32.
    """
    lib = load()
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a [B, T, D] tensor")
    B, T, D = x.shape
    dt, W, params = _conv_params(x, weight, bias, activation)
    xp, ldx = _rows(x, "x", x.shape, x.dtype, x)
    cup, n_seqs, N = _sequences(cu_seqlens, B, x)
    dyp = _tensor(d_y, "d_y", x.shape, x.dtype, x)
    if dyp is None:
        raise TypeError("d_y must be a torch.Tensor")
    shape = (N, W - 1, D)
    h0 = _tensor(initial_state, "initial_state", shape, x.dtype, x)
    dx = torch.empty_like(d_y)
    dw = torch.empty((D, W), dtype=_F32, device=x.device)
    db = None if bias is None else torch.empty(D, dtype=_F32, device=x.device)
    dh0 = None if initial_state is None else torch.empty(shape, dtype=x.dtype, device=x.device)
    ws, ws_bytes, workspace = _workspace(workspace, short_conv_workspace_size(B, T, D, W), x)
    _check(lib.gdn_short_conv_bwd(xp, *params, h0, dyp, _tensor(d_final_state, "d_final_state", shape, x.dtype, x), cup,
                                  n_seqs, dx.data_ptr(), dw.data_ptr(), None if db is None else db.data_ptr(),
                                  None if dh0 is None else dh0.data_ptr(), B, T, D, W, ldx, dt, ws, ws_bytes,
                                  _stream(x)))
    return dx, dw, db, dh0


@_on_stream
def gdn_short_conv_step(x, state, weight, bias=None, activation="silu", state_out=None, y=None):
    """One decode token of the short convolution for N sequences (C ABI gdn_short_conv_step); returns y [N, D].

    ``state`` [N, W - 1, D] in x's type moves up by the token in place, or is kept when ``state_out`` is given.
    """
    lib = load()
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be an [N, D] tensor")
    N, D = x.shape
    dt, W, params = _conv_params(x, weight, bias, activation)
    xp, ldx = _rows(x, "x", x.shape, x.dtype, x)
    shape = (N, W - 1, D)
    sp = _tensor(state, "state", shape, x.dtype, x)
    if y is None:
        y = torch.empty((N, D), dtype=x.dtype, device=x.device)
    _check(lib.gdn_short_conv_step(xp, *params, sp,
                                   sp if state_out is None else _tensor(state_out, "state_out", shape, x.dtype, x),
                                   _tensor(y, "y", x.shape, x.dtype, x), N, D, W, ldx, dt, _stream(x)))
    return y
