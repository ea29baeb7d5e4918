"""ctypes declarations of libgdn.so (the C ABI of include/gdn.h).

Loading fails loudly when the library has not been built: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn.so")

VERSION = 400   # GDN_VERSION of the header that these declarations follow

GDN_OK, GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED, GDN_ERR_CUDA, GDN_ERR_TIMEOUT, GDN_ERR_WORKSPACE = range(6)
GDN_F32, GDN_BF16 = 0, 1
GDN_NORMALIZE_QK = 0x1
GDN_RAW_GATES = 0x2
GDN_OUTPUT_GATE = 0x4

EXPORTED = ("gdn_opts_init", "gdn_chunk_fwd", "gdn_chunk_fwd_workspace_size", "gdn_recurrent_step",
            "gdn_check_device_status", "gdn_status_string", "gdn_last_error", "gdn_version",
            "gdn_chunk_fwd_noalloc", "gdn_causal_conv1d_fwd", "gdn_causal_conv1d_step",
            "gdn_recurrent_bwd", "gdn_recurrent_bwd_workspace_size", "gdn_causal_conv1d_fwd_qkv",
            "gdn_causal_conv1d_step_qkv", "gdn_output_gate_fwd", "gdn_output_gate_bwd",
            "gdn_output_gate_bwd_workspace_size", "gdn_causal_conv1d_bwd", "gdn_causal_conv1d_bwd_workspace_size",
            "gdn_decay_attn_fwd", "gdn_decay_attn_fwd_workspace_size", "gdn_decay_attn_step", "gdn_decay_attn_bwd",
            "gdn_decay_attn_bwd_workspace_size", "gdn_block_norm_fwd", "gdn_block_norm_bwd",
            "gdn_block_norm_bwd_workspace_size", "gdn_selective_scan_fwd", "gdn_selective_scan_fwd_workspace_size",
            "gdn_selective_scan_step", "gdn_selective_scan_bwd", "gdn_selective_scan_bwd_workspace_size",
            "gdn_layer_norm_fwd", "gdn_layer_norm_bwd", "gdn_layer_norm_bwd_workspace_size")


class GdnOpts(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int),
        ("chunk", ctypes.c_int),
        ("scale", ctypes.c_float),
        ("flags", ctypes.c_uint),
        ("cu_seqlens", ctypes.c_void_p),
        ("num_seqs", ctypes.c_int),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("stream", ctypes.c_void_p),
        ("events", ctypes.POINTER(ctypes.c_void_p)),
        ("num_events", ctypes.c_int),
        ("A_log", ctypes.c_void_p),
        ("dt_bias", ctypes.c_void_p),
        ("z", ctypes.c_void_p),
        ("norm_weight", ctypes.c_void_p),
        ("norm_eps", ctypes.c_float),
        ("grad_A_log", ctypes.c_void_p),
        ("grad_dt_bias", ctypes.c_void_p),
        ("conv_bias", ctypes.c_void_p),
        ("grad_conv_bias", ctypes.c_void_p),
    ]


class GdnError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"libgdn status {status}: {message}")
        self.status = status


_lib = None


def load(path: str = LIB_PATH):
    """Load libgdn.so and declare its entry points (cached)."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"libgdn.so is not built ({path}); run __graft_entry__.build() "
                          "or python -m gated_deltanet_recurrence_03_gb300.build")
    lib = ctypes.CDLL(path)
    lib.gdn_version.argtypes = []
    lib.gdn_version.restype = ctypes.c_int
    if lib.gdn_version() // 100 != VERSION // 100:   # another layout of GdnOpts
        raise ImportError(f"{path} is version {lib.gdn_version()}, these declarations are of {VERSION}; run "
                          "__graft_entry__.build() or python -m gated_deltanet_recurrence_03_gb300.build")
    vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    opts_p = ctypes.POINTER(GdnOpts)
    lib.gdn_opts_init.argtypes = [opts_p]
    lib.gdn_opts_init.restype = None
    lib.gdn_chunk_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, opts_p]
    lib.gdn_chunk_fwd.restype = i
    lib.gdn_chunk_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, opts_p]
    lib.gdn_chunk_fwd_noalloc.restype = i
    ll = ctypes.c_longlong
    lib.gdn_causal_conv1d_fwd.argtypes = [vp, ll, vp, vp, vp, vp, i, i, i, i, opts_p]
    lib.gdn_causal_conv1d_fwd.restype = i
    lib.gdn_causal_conv1d_step.argtypes = [vp, ll, vp, vp, vp, i, i, i, opts_p]
    lib.gdn_causal_conv1d_step.restype = i
    lib.gdn_causal_conv1d_fwd_qkv.argtypes = [vp, ll, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, opts_p]
    lib.gdn_causal_conv1d_fwd_qkv.restype = i
    lib.gdn_causal_conv1d_step_qkv.argtypes = [vp, ll, vp, vp, vp, vp, vp, i, i, i, i, i, opts_p]
    lib.gdn_causal_conv1d_step_qkv.restype = i
    lib.gdn_recurrent_bwd.argtypes = [vp] * 14 + [i, i, i, i, i, i, opts_p]
    lib.gdn_recurrent_bwd.restype = i
    lib.gdn_output_gate_fwd.argtypes = [vp, vp, vp, vp, ll, i, opts_p]
    lib.gdn_output_gate_fwd.restype = i
    lib.gdn_output_gate_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, ll, i, opts_p]
    lib.gdn_output_gate_bwd.restype = i
    lib.gdn_output_gate_bwd_workspace_size.argtypes = [ll, i, opts_p]
    lib.gdn_output_gate_bwd_workspace_size.restype = ctypes.c_size_t
    lib.gdn_causal_conv1d_bwd.argtypes = [vp, ll, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, opts_p]
    lib.gdn_causal_conv1d_bwd.restype = i
    lib.gdn_causal_conv1d_bwd_workspace_size.argtypes = [i, i, i, i, opts_p]
    lib.gdn_causal_conv1d_bwd_workspace_size.restype = ctypes.c_size_t
    lib.gdn_recurrent_bwd_workspace_size.argtypes = [i, i, i, i, i, i, opts_p]
    lib.gdn_recurrent_bwd_workspace_size.restype = ctypes.c_size_t
    lib.gdn_chunk_fwd_workspace_size.argtypes = [i, i, i, i, i, i, opts_p]
    lib.gdn_chunk_fwd_workspace_size.restype = ctypes.c_size_t
    lib.gdn_recurrent_step.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, opts_p]
    lib.gdn_recurrent_step.restype = i
    lib.gdn_decay_attn_fwd.argtypes = [vp, ll, vp, ll, vp, ll, vp, vp, vp, vp, i, i, i, i, i, i, opts_p]
    lib.gdn_decay_attn_fwd.restype = i
    lib.gdn_decay_attn_step.argtypes = [vp, ll, vp, ll, vp, ll, vp, vp, vp, i, vp, i, i, i, i, i, opts_p]
    lib.gdn_decay_attn_step.restype = i
    lib.gdn_decay_attn_bwd.argtypes = [vp, ll, vp, ll, vp, ll, vp, vp, vp, vp, vp, ll, vp, ll, vp, ll, vp,
                                       i, i, i, i, i, i, opts_p]
    lib.gdn_decay_attn_bwd.restype = i
    for size in (lib.gdn_decay_attn_fwd_workspace_size, lib.gdn_decay_attn_bwd_workspace_size):
        size.argtypes = [i, i, i, i, i, i, opts_p]
        size.restype = ctypes.c_size_t
    lib.gdn_block_norm_fwd.argtypes = [vp, vp, vp, i, vp, vp, vp, vp, vp, ll, i, opts_p]
    lib.gdn_block_norm_fwd.restype = i
    lib.gdn_block_norm_bwd.argtypes = [vp, vp, vp, i] + [vp] * 11 + [ll, i, opts_p]
    lib.gdn_block_norm_bwd.restype = i
    lib.gdn_block_norm_bwd_workspace_size.argtypes = [ll, i, opts_p]
    lib.gdn_block_norm_bwd_workspace_size.restype = ctypes.c_size_t
    scan_in = [vp, ll, vp, ll, vp, vp, ll, vp, ll, vp, vp, vp, ll]   # u, delta, A_log, B, C, skip, dt_bias, z
    lib.gdn_selective_scan_fwd.argtypes = scan_in + [vp] * 3 + [i] * 5 + [opts_p]
    lib.gdn_selective_scan_fwd.restype = i
    lib.gdn_selective_scan_step.argtypes = scan_in + [vp, vp, i, vp] + [i] * 4 + [opts_p]
    lib.gdn_selective_scan_step.restype = i
    lib.gdn_selective_scan_bwd.argtypes = (scan_in + [vp] * 7 + [ll, vp, ll, vp, vp, vp, ll, vp] + [i] * 5 + [opts_p])
    lib.gdn_selective_scan_bwd.restype = i
    for size in (lib.gdn_selective_scan_fwd_workspace_size, lib.gdn_selective_scan_bwd_workspace_size):
        size.argtypes = [i] * 5 + [opts_p]
        size.restype = ctypes.c_size_t
    lib.gdn_layer_norm_fwd.argtypes = [vp] * 6 + [ll, i, opts_p]
    lib.gdn_layer_norm_fwd.restype = i
    lib.gdn_layer_norm_bwd.argtypes = [vp] * 8 + [ll, i, opts_p]
    lib.gdn_layer_norm_bwd.restype = i
    lib.gdn_layer_norm_bwd_workspace_size.argtypes = [ll, i, opts_p]
    lib.gdn_layer_norm_bwd_workspace_size.restype = ctypes.c_size_t
    lib.gdn_check_device_status.argtypes = [vp]
    lib.gdn_check_device_status.restype = i
    lib.gdn_status_string.argtypes = [i]
    lib.gdn_status_string.restype = ctypes.c_char_p
    lib.gdn_last_error.argtypes = []
    lib.gdn_last_error.restype = ctypes.c_char_p
    if path == LIB_PATH:
        _lib = lib
    return lib


def check(lib, status: int) -> None:
    if status != GDN_OK:
        msg = lib.gdn_last_error().decode() or lib.gdn_status_string(status).decode()
        raise GdnError(status, msg)


def default_opts(lib) -> GdnOpts:
    o = GdnOpts()
    lib.gdn_opts_init(ctypes.byref(o))
    return o


_default_bytes = None


def default_bytes(lib) -> bytes:
    """default_opts as bytes (cached): options of a call are copied from it."""
    global _default_bytes
    if _default_bytes is None:
        _default_bytes = bytes(default_opts(lib))
    return _default_bytes
