"""GB300-native (sm_103a) gated delta rule: chunkwise forward and backward, KDA, and the decode step; and the operators
around it: the short convolution, the query/key head norm with rotation, and the gated linear recurrence.

The computation lives in libgdn_gb300.so (C ABI, include/gdn.h): hand-written
CUDA kernels for sm_103a.  This package is its thin Python binding (ctypes,
and an extension module for the entry points that _mixer.py lists); torch
supplies device memory and streams.  Build the library with
``gated_delta_rule_gdn_gb300.build.build()``; the calls raise if it is
missing.
"""
from ._binding import (GdnError, bwd_workspace_size, chunk_bwd, chunk_fwd_noalloc, gdn_chunk_bwd, kda_chunk_bwd, chunk_plan, device_status, gdn_chunk_fwd, gdn_recurrent_step, kda_chunk_fwd, kda_recurrent_step, last_error,
                       lib_path, load, workspace_size)
from . import _mixer
from ._mixer import glr_workspace_size, qk_norm_workspace_size, short_conv_workspace_size

__all__ = ["gdn_chunk_fwd", "kda_chunk_fwd", "gdn_recurrent_step", "kda_recurrent_step", "device_status", "chunk_plan", "last_error", "load",
           "lib_path", "GdnError", "workspace_size", "chunk_fwd_noalloc",
           "chunk_bwd", "gdn_chunk_bwd", "kda_chunk_bwd", "bwd_workspace_size",
           "gdn_short_conv_fwd", "gdn_short_conv_bwd", "gdn_short_conv_step", "short_conv_workspace_size",
           "gdn_qk_norm_fwd", "gdn_qk_norm_bwd", "qk_norm_workspace_size",
           "glr_scan_fwd", "glr_scan_bwd", "glr_step", "glr_workspace_size"]


def __getattr__(name):
    """The entry points of the extension module, which is loaded when the first of them is asked for (before it is built,
    they raise when called)."""
    if name not in _mixer.ENTRIES:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    if not _mixer.built():
        return lambda *args, **kw: getattr(_mixer.native(), name)(*args, **kw)
    globals()[name] = entry = getattr(_mixer.native(), name)
    return entry
