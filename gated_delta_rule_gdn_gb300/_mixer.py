"""Binding of the operators around the delta rule (the gated linear recurrence, the query/key head norm with rotation, the
short causal convolution) and beside it (linear attention with a decay for each head, the paged key-value cache).

The entry points themselves are in the extension module _native (csrc/torch_binding.cpp), which checks the tensors,
allocates outputs and workspaces, and calls the C ABI; see their docstrings.  Inputs may be cut out of a wider projection
(their rows must be contiguous and evenly spaced); outputs are contiguous.  Calls run on the current stream, or on
``stream``; with ``stream`` their outputs and workspaces are allocated on it too, so that the allocator does not hand
their memory to other streams while the call runs.  Inputs, and buffers that are handed in, are the caller's to have ready
on that stream and to keep until its work is done, as for any torch operation on a stream that is not the tensors' own.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

from . import build as _build
from ._binding import _check, load

ENTRIES = ("glr_scan_fwd", "glr_scan_bwd", "glr_step", "gdn_qk_norm_fwd", "gdn_qk_norm_bwd", "gdn_short_conv_fwd",
           "gdn_short_conv_bwd", "gdn_short_conv_step", "lin_chunk_fwd", "lin_chunk_bwd", "lin_recurrent_step", "paged_append",
           "paged_attn_step")
_SIZES = ("glr_workspace_size", "gdn_qk_norm_workspace_size", "gdn_short_conv_workspace_size", "lin_workspace_size",
          "paged_attn_workspace_size")

_NATIVE = None


def declare(lib):
    """Argument types of the entry points (called once, when the library is loaded)."""
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
        "lin_chunk_fwd": [vp] * 4 + [i, fp, vp, vp, vp, i, vp] + [i] * 6 + [i64] * 6 + [i, i, vp, sz, vp],
        "lin_chunk_bwd": [vp] * 4 + [i, fp] + [vp] * 4 + [i] + [vp] * 5 + [i] * 6 + [i64] * 6 + [i, i, vp, sz, vp],
        "lin_workspace_size": [i] * 8 + [szp],
        "lin_recurrent_step": [vp] * 4 + [i, fp, vp, vp, vp] + [i] * 5 + [i64] * 6 + [i, vp],
        "paged_append": [vp] * 7 + [i, i, i, vp, i64, i] + [i64] * 6 + [vp],
        "paged_attn_step": [vp, vp, fp, vp, vp, i, i64, i64, vp, sz, vp],
        "paged_attn_workspace_size": [i] * 6 + [szp],
    }.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = i, args


def built() -> bool:
    return os.path.exists(_build.LIB) and os.path.exists(_build.NATIVE)


def native():
    """The extension module, bound to the library's entry points; raises if it is not built."""
    global _NATIVE
    if _NATIVE is None:
        lib, path = load(), _build.NATIVE
        if not os.path.exists(path):
            raise RuntimeError(f"the binding is not built ({path}); run "
                               "`python -c 'import __graft_entry__ as g; g.build()'` first")
        if not _build.native_current():
            raise RuntimeError(f"the binding ({path}) was built with another torch or Python; run "
                               "`python -c 'import __graft_entry__ as g; g.build()'` again")
        loader = importlib.machinery.ExtensionFileLoader("_native", path)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_native", loader))
        loader.exec_module(module)
        module.init(_check, {n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in ENTRIES + _SIZES})
        _NATIVE = module
    return _NATIVE


def glr_workspace_size(B: int, T: int, D: int, n_seqs: int = 0, backward: bool = False) -> int:
    """Device workspace bytes of glr_scan_fwd, or glr_scan_bwd (C ABI glr_workspace_size)."""
    out = ctypes.c_size_t(0)
    _check(load().glr_workspace_size(int(backward), B, T, D, n_seqs, ctypes.byref(out)))
    return out.value


def qk_norm_workspace_size(n_tokens: int, H_q: int, H_k: int, d: int) -> int:
    """Device workspace bytes of gdn_qk_norm_bwd (C ABI gdn_qk_norm_workspace_size)."""
    out = ctypes.c_size_t(0)
    _check(load().gdn_qk_norm_workspace_size(n_tokens, H_q, H_k, d, ctypes.byref(out)))
    return out.value


def short_conv_workspace_size(B: int, T: int, D: int, W: int) -> int:
    """Device workspace bytes of gdn_short_conv_bwd (C ABI gdn_short_conv_workspace_size)."""
    out = ctypes.c_size_t(0)
    _check(load().gdn_short_conv_workspace_size(B, T, D, W, ctypes.byref(out)))
    return out.value


def lin_workspace_size(B: int, T: int, H_k: int, H: int, d_k: int, d_v: int, n_seqs: int = 0, backward: bool = False) -> int:
    """Device workspace bytes of lin_chunk_fwd, or lin_chunk_bwd (C ABI lin_workspace_size)."""
    out = ctypes.c_size_t(0)
    _check(load().lin_workspace_size(int(backward), B, T, H_k, H, d_k, d_v, n_seqs, ctypes.byref(out)))
    return out.value


def paged_attn_workspace_size(N: int, H_q: int, H_k: int, d: int, max_pages: int, page_size: int) -> int:
    """Device workspace bytes of paged_attn_step (C ABI paged_attn_workspace_size)."""
    out = ctypes.c_size_t(0)
    _check(load().paged_attn_workspace_size(N, H_q, H_k, d, max_pages, page_size, ctypes.byref(out)))
    return out.value
