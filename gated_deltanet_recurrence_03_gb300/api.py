"""PyTorch-facing binding of libgdn: argument marshalling only.

Each function checks shapes and dtypes, allocates the outputs (and the scratch
workspace) with PyTorch, and calls the C ABI entry point of the same name on the
current (or given) CUDA stream.  Every step of the recurrence runs in libgdn's
CUDA kernels; there is no other code path.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional, Sequence

import torch

from . import _lib as L

_DTYPES = {torch.float32: L.GDN_F32, torch.bfloat16: L.GDN_BF16}


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _need(name, t, dtype, device, shape):
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _stream_handle(stream: Optional[torch.cuda.Stream], device) -> int:
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return int(s.cuda_stream)


_NO_SWITCH = contextlib.nullcontext()
_DENSE = torch.contiguous_format   # empty_like of a slice is dense (and 1 to 2 us cheaper than new_empty)


def _on(device, stream=None):
    """Context in which ``device`` and, where given, ``stream`` are current; costs nothing where they already are.
    What a call allocates in it belongs to the stream that its kernels run on, so that neither memory still in use
    on another stream is written nor the call's own handed out before it is done."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
        return torch.cuda.stream(stream)
    return _NO_SWITCH if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def _call_opts(lib, dtype, scale, stream, device, events):
    """Options of a call without flags: the library's defaults with the type, scale, stream and events."""
    o = L.GdnOpts.from_buffer_copy(L.default_bytes(lib))
    o.dtype = _DTYPES[dtype]
    o.scale = scale
    o.stream = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(device.index)
    keep = None
    if events:
        keep = (ctypes.c_void_p * len(events))(*[int(e) for e in events])
        o.events = ctypes.cast(keep, ctypes.POINTER(ctypes.c_void_p))
        o.num_events = len(events)
    return o, keep


def _opts(lib, dtype, scale, chunk, normalize_qk, stream, device, events, raw_gates=None, Hv=None,
          output_gate=None, out_shape=None):
    o = L.default_opts(lib)
    o.dtype = _DTYPES[dtype]
    o.chunk = int(chunk)
    o.scale = float(scale)
    o.flags = L.GDN_NORMALIZE_QK if normalize_qk else 0
    if raw_gates is not None:
        A_log, dt_bias = raw_gates
        _need("A_log", A_log, torch.float32, device, (Hv,))
        _need("dt_bias", dt_bias, torch.float32, device, (Hv,))
        o.flags |= L.GDN_RAW_GATES
        o.A_log = A_log.data_ptr()
        o.dt_bias = dt_bias.data_ptr()
    if output_gate is not None:
        z, weight, eps = output_gate
        _need("z", z, dtype, device, out_shape)
        _need("norm_weight", weight, torch.float32, device, (out_shape[-1],))
        o.flags |= L.GDN_OUTPUT_GATE
        o.z = z.data_ptr()
        o.norm_weight = weight.data_ptr()
        o.norm_eps = float(eps)
    o.stream = _stream_handle(stream, device)
    keep = None
    if events:
        keep = (ctypes.c_void_p * len(events))(*[int(e) for e in events])
        o.events = ctypes.cast(keep, ctypes.POINTER(ctypes.c_void_p))
        o.num_events = len(events)
    return o, keep


def workspace_size(B: int, T: int, Hqk: int, Hv: int, dk: int, dv: int, *, dtype=torch.bfloat16,
                   chunk: int = 64, num_seqs: Optional[int] = None) -> int:
    """Bytes of device scratch gdn_chunk_fwd needs (0 when the selected kernel needs none)."""
    lib = L.load()
    o = L.default_opts(lib)
    o.dtype = _DTYPES[dtype]
    o.chunk = int(chunk)
    if num_seqs is not None:
        o.cu_seqlens = 16  # any non-null value marks the call as packed for the size query
        o.num_seqs = int(num_seqs)
    return int(lib.gdn_chunk_fwd_workspace_size(B, T, Hqk, Hv, dk, dv, ctypes.byref(o)))


def gdn_chunk_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                  S0: Optional[torch.Tensor] = None, *, scale: float = 1.0, chunk: int = 64,
                  normalize_qk: bool = False, cu_seqlens: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, S_final: Optional[torch.Tensor] = None,
                  output_final_state: bool = True, workspace: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None, events: Optional[Sequence[int]] = None,
                  raw_gates=None, output_gate=None):
    """Chunked prefill.  q, k [B, T, Hqk, dk]; v [B, T, Hv, dv]; g, beta [B, T, Hv] (all bf16 or all
    fp32, on one CUDA device); S0 [nseq, Hv, dk, dv] fp32 or None.  With ``cu_seqlens`` (int32 device
    tensor of nseq+1 offsets) B must be 1.  With ``raw_gates=(A_log, dt_bias)`` (fp32 [Hv] each), g and
    beta are the raw projections a and b and the kernels form the gates.  With
    ``output_gate=(z, norm_weight, eps)`` (z like out, norm_weight fp32 [dv]) the outputs pass through
    RMSNorm * norm_weight * silu(z).  Returns (out [B, T, Hv, dv], S_final or None)."""
    lib = L.load()
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be 4-D [B, T, H, d]")
    B, T, Hqk, dk = q.shape
    Hv, dv = int(v.shape[2]), int(v.shape[3])
    dev, dt = q.device, q.dtype
    if dt not in _DTYPES:
        raise ValueError(f"unsupported dtype {dt}")
    _need("q", q, dt, dev, (B, T, Hqk, dk))
    _need("k", k, dt, dev, (B, T, Hqk, dk))
    _need("v", v, dt, dev, (B, T, Hv, dv))
    _need("g", g, dt, dev, (B, T, Hv))
    _need("beta", beta, dt, dev, (B, T, Hv))
    nseq = B
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1:
            raise ValueError("cu_seqlens must be 1-D")
        nseq = int(cu_seqlens.numel()) - 1
        _need("cu_seqlens", cu_seqlens, torch.int32, dev, (nseq + 1,))
    if S0 is not None:
        _need("S0", S0, torch.float32, dev, (nseq, Hv, dk, dv))
    if out is None:
        out = torch.empty_like(v)
    _need("out", out, dt, dev, (B, T, Hv, dv))
    if S_final is None and output_final_state:
        S_final = torch.empty((nseq, Hv, dk, dv), dtype=torch.float32, device=dev)
    if S_final is not None:
        _need("S_final", S_final, torch.float32, dev, (nseq, Hv, dk, dv))
    with torch.cuda.device(dev):
        o, keep = _opts(lib, dt, scale, chunk, normalize_qk, stream, dev, events, raw_gates, Hv,
                        output_gate, (B, T, Hv, dv))
        if cu_seqlens is not None:
            o.cu_seqlens = cu_seqlens.data_ptr()
            o.num_seqs = nseq
        need = int(lib.gdn_chunk_fwd_workspace_size(B, T, Hqk, Hv, dk, dv, ctypes.byref(o)))
        if need:
            if workspace is None or workspace.numel() * workspace.element_size() < need:
                workspace = torch.empty(need, dtype=torch.uint8, device=dev)
            o.workspace = workspace.data_ptr()
            o.workspace_bytes = workspace.numel() * workspace.element_size()
        st = lib.gdn_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S0), _ptr(out),
                               _ptr(S_final), B, T, Hqk, Hv, dk, dv, ctypes.byref(o))
        del keep
        L.check(lib, st)
    return out, S_final


def gdn_recurrent_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                       S: torch.Tensor, *, scale: float = 1.0, normalize_qk: bool = False,
                       out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None,
                       events: Optional[Sequence[int]] = None, raw_gates=None,
                       output_gate=None) -> torch.Tensor:
    """One decode step.  q, k [N, Hqk, dk]; v [N, Hv, dv]; g, beta [N, Hv]; S [N, Hv, dk, dv] fp32 is
    updated in place.  ``raw_gates`` and ``output_gate`` as for gdn_chunk_fwd.  Returns out [N, Hv, dv]."""
    lib = L.load()
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k, v must be 3-D [N, H, d]")
    N, Hqk, dk = q.shape
    Hv, dv = int(v.shape[1]), int(v.shape[2])
    dev, dt = q.device, q.dtype
    if dt not in _DTYPES:
        raise ValueError(f"unsupported dtype {dt}")
    _need("q", q, dt, dev, (N, Hqk, dk))
    _need("k", k, dt, dev, (N, Hqk, dk))
    _need("v", v, dt, dev, (N, Hv, dv))
    _need("g", g, dt, dev, (N, Hv))
    _need("beta", beta, dt, dev, (N, Hv))
    _need("S", S, torch.float32, dev, (N, Hv, dk, dv))
    if out is None:
        out = torch.empty_like(v)
    _need("out", out, dt, dev, (N, Hv, dv))
    with torch.cuda.device(dev):
        o, keep = _opts(lib, dt, scale, 64, normalize_qk, stream, dev, events, raw_gates, Hv,
                        output_gate, (N, Hv, dv))
        st = lib.gdn_recurrent_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S), _ptr(out),
                                    N, Hqk, Hv, dk, dv, ctypes.byref(o))
        del keep
        L.check(lib, st)
    return out


def check_device_status(stream: Optional[torch.cuda.Stream] = None, device=None) -> None:
    """Synchronise and raise GdnError if a kernel reported a bounded wait that ran out."""
    lib = L.load()
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        L.check(lib, lib.gdn_check_device_status(_stream_handle(stream, dev)))


def version() -> int:
    return int(L.load().gdn_version())


def _conv_bias(o, bias, C, dev):
    if bias is not None:
        _need("bias", bias, torch.float32, dev, (C,))
        o.conv_bias = bias.data_ptr()


def gdn_causal_conv1d_fwd(x: torch.Tensor, w: torch.Tensor, cache_in: Optional[torch.Tensor] = None, *,
                          bias: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
                          out: Optional[torch.Tensor] = None,
                          cache_out: Optional[torch.Tensor] = None, return_cache: bool = True, stream: Optional[torch.cuda.Stream] = None,
                          events: Optional[Sequence[int]] = None):
    """Depthwise causal convolution + SiLU.  x [B, T, C] (bf16 or fp32; may be a channel slice of a
    wider tensor: rows must be evenly strided with the channels contiguous); w [C, K] fp32;
    cache_in [nseq, K-1, C] or None.  ``cache_out`` (or a new tensor when ``return_cache``) receives each
    sequence's last K-1 inputs.  ``bias`` (fp32 [C] or None) is added before the SiLU.  Returns (y [B, T, C],
    cache_out [nseq, K-1, C] or None)."""
    lib = L.load()
    if x.dim() != 3 or x.stride(2) != 1 or x.stride(0) != x.shape[1] * x.stride(1):
        raise ValueError("x must be [B, T, C] with contiguous channels and evenly strided token rows")
    B, T, C = x.shape
    dev, dt = x.device, x.dtype
    if dt not in _DTYPES:
        raise ValueError(f"unsupported dtype {dt}")
    K = int(w.shape[1])
    _need("w", w, torch.float32, dev, (C, K))
    nseq = B
    if cu_seqlens is not None:
        nseq = int(cu_seqlens.numel()) - 1
        _need("cu_seqlens", cu_seqlens, torch.int32, dev, (nseq + 1,))
    if cache_in is not None:
        _need("cache_in", cache_in, dt, dev, (nseq, K - 1, C))
    with _on(dev, stream):
        if out is None:
            out = torch.empty((B, T, C), dtype=dt, device=dev)
        _need("out", out, dt, dev, (B, T, C))
        if cache_out is None and return_cache:
            cache_out = torch.empty((nseq, K - 1, C), dtype=dt, device=dev)
        if cache_out is not None:
            _need("cache_out", cache_out, dt, dev, (nseq, K - 1, C))
        o, keep = _opts(lib, dt, 1.0, 64, False, stream, dev, events)
        if cu_seqlens is not None:
            o.cu_seqlens = cu_seqlens.data_ptr()
            o.num_seqs = nseq
        _conv_bias(o, bias, C, dev)
        st = lib.gdn_causal_conv1d_fwd(_ptr(x), x.stride(1), _ptr(w), _ptr(cache_in), _ptr(out), _ptr(cache_out),
                                       B, T, C, K, ctypes.byref(o))
        del keep
        L.check(lib, st)
    return out, cache_out


def gdn_causal_conv1d_bwd(x: torch.Tensor, w: torch.Tensor, grad_y: torch.Tensor, cache_in: Optional[torch.Tensor] = None,
                          *, bias: Optional[torch.Tensor] = None, grad_cache_out: Optional[torch.Tensor] = None,
                          cu_seqlens: Optional[torch.Tensor] = None, want_grad_w: bool = True,
                          want_grad_cache_in: bool = True, stream: Optional[torch.cuda.Stream] = None,
                          events: Optional[Sequence[int]] = None):
    """Gradients through gdn_causal_conv1d_fwd: x, w, cache_in, bias as there; grad_y [B, T, C] like x (dense);
    grad_cache_out [nseq, K-1, C] like x or None.  Returns fp32 (grad_x [B, T, C], grad_w [C, K] or None,
    grad_cache_in [nseq, K-1, C] or None), and with a bias a fourth one, grad_bias [C]."""
    lib = L.load()
    if x.dim() != 3 or x.stride(2) != 1 or x.stride(0) != x.shape[1] * x.stride(1):
        raise ValueError("x must be [B, T, C] with contiguous channels and evenly strided token rows")
    B, T, C = x.shape
    dev, dt = x.device, x.dtype
    if dt not in _DTYPES:
        raise ValueError(f"unsupported dtype {dt}")
    K = int(w.shape[1])
    _need("w", w, torch.float32, dev, (C, K))
    _need("grad_y", grad_y, dt, dev, (B, T, C))
    nseq = B
    if cu_seqlens is not None:
        nseq = int(cu_seqlens.numel()) - 1
        _need("cu_seqlens", cu_seqlens, torch.int32, dev, (nseq + 1,))
    if cache_in is not None:
        _need("cache_in", cache_in, dt, dev, (nseq, K - 1, C))
    if grad_cache_out is not None:
        _need("grad_cache_out", grad_cache_out, dt, dev, (nseq, K - 1, C))
    f32 = dict(dtype=torch.float32, device=dev)
    with _on(dev, stream):
        gx = torch.empty((B, T, C), **f32)
        gw = torch.empty((C, K), **f32) if want_grad_w else None
        gc = torch.empty((nseq, K - 1, C), **f32) if want_grad_cache_in and K > 1 else None
        o, keep = _opts(lib, dt, 1.0, 64, False, stream, dev, events)
        if cu_seqlens is not None:
            o.cu_seqlens = cu_seqlens.data_ptr()
            o.num_seqs = nseq
        _conv_bias(o, bias, C, dev)
        gb = None
        if bias is not None:
            gb = (torch.empty if nseq > 0 else torch.zeros)((C,), **f32)   # no sequences: nothing is launched
            o.grad_conv_bias = gb.data_ptr()
        ws = None
        if want_grad_w or gb is not None:
            need = int(lib.gdn_causal_conv1d_bwd_workspace_size(B, T, C, K, ctypes.byref(o)))
            ws = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
            o.workspace, o.workspace_bytes = ws.data_ptr(), ws.numel()
        st = lib.gdn_causal_conv1d_bwd(_ptr(x), x.stride(1), _ptr(w), _ptr(cache_in), _ptr(grad_y),
                                       _ptr(grad_cache_out), _ptr(gx), _ptr(gw), _ptr(gc), B, T, C, K,
                                       ctypes.byref(o))
        del keep
        L.check(lib, st)
    return (gx, gw, gc) if bias is None else (gx, gw, gc, gb)


def gdn_causal_conv1d_step(x: torch.Tensor, w: torch.Tensor, cache: torch.Tensor, *,
                           bias: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                           stream: Optional[torch.cuda.Stream] = None,
                           events: Optional[Sequence[int]] = None) -> torch.Tensor:
    """One decode token per sequence: x [N, C] (channels contiguous, rows evenly strided), w [C, K] fp32,
    cache [N, K-1, C] updated in place; bias fp32 [C] or None.  Returns y [N, C]."""
    lib = L.load()
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be [N, C] with contiguous channels")
    N, C = x.shape
    dev, dt = x.device, x.dtype
    K = int(w.shape[1])
    _need("w", w, torch.float32, dev, (C, K))
    _need("cache", cache, dt, dev, (N, K - 1, C))
    with _on(dev, stream):
        if out is None:
            out = torch.empty((N, C), dtype=dt, device=dev)
        _need("out", out, dt, dev, (N, C))
        o, keep = _opts(lib, dt, 1.0, 64, False, stream, dev, events)
        _conv_bias(o, bias, C, dev)
        st = lib.gdn_causal_conv1d_step(_ptr(x), x.stride(0), _ptr(w), _ptr(cache), _ptr(out), N, C, K,
                                        ctypes.byref(o))
        del keep
        L.check(lib, st)
    return out


def gdn_causal_conv1d_fwd_qkv(x: torch.Tensor, w: torch.Tensor, widths: Sequence[int],
                              cache_in: Optional[torch.Tensor] = None, *, bias: Optional[torch.Tensor] = None,
                              cu_seqlens: Optional[torch.Tensor] = None, out: Optional[Sequence[torch.Tensor]] = None,
                              cache_out: Optional[torch.Tensor] = None,
                              return_cache: bool = True, stream: Optional[torch.cuda.Stream] = None,
                              events: Optional[Sequence[int]] = None):
    """The convolution of gdn_causal_conv1d_fwd over the packed q | k | v projection x [B, T, Cq + Ck + Cv]
    in one launch, the three channel ranges (``widths`` = (Cq, Ck, Cv)) written to three dense tensors.
    Returns ((y_q, y_k, y_v), cache_out [nseq, K-1, C] or None)."""
    lib = L.load()
    if x.dim() != 3 or x.stride(2) != 1 or x.stride(0) != x.shape[1] * x.stride(1):
        raise ValueError("x must be [B, T, C] with contiguous channels and evenly strided token rows")
    B, T, C = x.shape
    Cq, Ck, Cv = (int(c) for c in widths)
    if Cq + Ck + Cv != C:
        raise ValueError(f"widths {widths} do not add up to the {C} channels of x")
    dev, dt = x.device, x.dtype
    if dt not in _DTYPES:
        raise ValueError(f"unsupported dtype {dt}")
    K = int(w.shape[1])
    _need("w", w, torch.float32, dev, (C, K))
    nseq = B
    if cu_seqlens is not None:
        nseq = int(cu_seqlens.numel()) - 1
        _need("cu_seqlens", cu_seqlens, torch.int32, dev, (nseq + 1,))
    if cache_in is not None:
        _need("cache_in", cache_in, dt, dev, (nseq, K - 1, C))
    with _on(dev, stream):
        if out is None:
            out = tuple(torch.empty((B, T, c), dtype=dt, device=dev) for c in (Cq, Ck, Cv))
        for name, y, c in zip(("y_q", "y_k", "y_v"), out, (Cq, Ck, Cv)):
            _need(name, y, dt, dev, (B, T, c))
        if cache_out is None and return_cache:
            cache_out = torch.empty((nseq, K - 1, C), dtype=dt, device=dev)
        if cache_out is not None:
            _need("cache_out", cache_out, dt, dev, (nseq, K - 1, C))
        o, keep = _opts(lib, dt, 1.0, 64, False, stream, dev, events)
        if cu_seqlens is not None:
            o.cu_seqlens = cu_seqlens.data_ptr()
            o.num_seqs = nseq
        _conv_bias(o, bias, C, dev)
        st = lib.gdn_causal_conv1d_fwd_qkv(_ptr(x), x.stride(1), _ptr(w), _ptr(cache_in), _ptr(out[0]), _ptr(out[1]),
                                           _ptr(out[2]), _ptr(cache_out), B, T, Cq, Ck, Cv, K, ctypes.byref(o))
        del keep
        L.check(lib, st)
    return tuple(out), cache_out


def gdn_causal_conv1d_step_qkv(x: torch.Tensor, w: torch.Tensor, cache: torch.Tensor, widths: Sequence[int], *,
                               bias: Optional[torch.Tensor] = None, out: Optional[Sequence[torch.Tensor]] = None,
                               stream: Optional[torch.cuda.Stream] = None,
                               events: Optional[Sequence[int]] = None):
    """One decode token per sequence through the convolution of the packed q | k | v projection
    x [N, Cq + Ck + Cv] (``widths`` = (Cq, Ck, Cv)), cache [N, K-1, C] updated in place, in one launch.
    Returns (y_q [N, Cq], y_k [N, Ck], y_v [N, Cv])."""
    lib = L.load()
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be [N, C] with contiguous channels")
    N, C = x.shape
    Cq, Ck, Cv = (int(c) for c in widths)
    if Cq + Ck + Cv != C:
        raise ValueError(f"widths {widths} do not add up to the {C} channels of x")
    dev, dt = x.device, x.dtype
    K = int(w.shape[1])
    _need("w", w, torch.float32, dev, (C, K))
    _need("cache", cache, dt, dev, (N, K - 1, C))
    with _on(dev, stream):
        if out is None:
            out = tuple(torch.empty((N, c), dtype=dt, device=dev) for c in (Cq, Ck, Cv))
        for name, y, c in zip(("y_q", "y_k", "y_v"), out, (Cq, Ck, Cv)):
            _need(name, y, dt, dev, (N, c))
        o, keep = _opts(lib, dt, 1.0, 64, False, stream, dev, events)
        _conv_bias(o, bias, C, dev)
        st = lib.gdn_causal_conv1d_step_qkv(_ptr(x), x.stride(0), _ptr(w), _ptr(cache), _ptr(out[0]), _ptr(out[1]),
                                            _ptr(out[2]), N, Cq, Ck, Cv, K, ctypes.byref(o))
        del keep
        L.check(lib, st)
    return tuple(out)


def backward_workspace_size(B: int, T: int, Hqk: int, Hv: int, dk: int, dv: int, *,
                            num_seqs: Optional[int] = None, front_end: bool = False) -> int:
    """Bytes of device scratch gdn_recurrent_bwd needs (with ``front_end``: through the l2 norm and / or
    the raw gates)."""
    lib = L.load()
    o = L.default_opts(lib)
    if front_end:
        o.flags = L.GDN_NORMALIZE_QK
    if num_seqs is not None:
        o.cu_seqlens = 1   # only tested for NULL
        o.num_seqs = int(num_seqs)
    return int(lib.gdn_recurrent_bwd_workspace_size(B, T, Hqk, Hv, dk, dv, ctypes.byref(o)))


def gdn_recurrent_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                      S0: Optional[torch.Tensor], grad_out: torch.Tensor, grad_S_final: Optional[torch.Tensor] = None,
                      *, scale: float = 1.0, cu_seqlens: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, want_grad_S0: bool = True,
                      stream: Optional[torch.cuda.Stream] = None, events: Optional[Sequence[int]] = None,
                      normalize_qk: bool = False, raw_gates=None):
    """Gradients of a loss on (out, S_final) of gdn_chunk_fwd with respect to q, k, v, g, beta, S0.
    Inputs as for gdn_chunk_fwd; grad_out like v; grad_S_final fp32 like S_final or None.  Returns fp32
    (grad_q, grad_k, grad_v, grad_g, grad_beta, grad_S0 or None).  With normalize_qk and / or
    raw_gates=(A_log, dt_bias) (g and beta then hold the raw projections a and b) the gradients are
    those of the forward with the same front end, with respect to its raw inputs, and two more tensors
    are returned with raw_gates: grad_A_log, grad_dt_bias (fp32 [Hv])."""
    lib = L.load()
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be 4-D [B, T, H, d]")
    B, T, Hqk, dk = q.shape
    Hv, dv = int(v.shape[2]), int(v.shape[3])
    dev, dt = q.device, q.dtype
    if dt not in _DTYPES:
        raise ValueError(f"unsupported dtype {dt}")
    _need("q", q, dt, dev, (B, T, Hqk, dk))
    _need("k", k, dt, dev, (B, T, Hqk, dk))
    _need("v", v, dt, dev, (B, T, Hv, dv))
    _need("g", g, dt, dev, (B, T, Hv))
    _need("beta", beta, dt, dev, (B, T, Hv))
    _need("grad_out", grad_out, dt, dev, (B, T, Hv, dv))
    nseq = B
    if cu_seqlens is not None:
        nseq = int(cu_seqlens.numel()) - 1
        _need("cu_seqlens", cu_seqlens, torch.int32, dev, (nseq + 1,))
    if S0 is not None:
        _need("S0", S0, torch.float32, dev, (nseq, Hv, dk, dv))
    if grad_S_final is not None:
        _need("grad_S_final", grad_S_final, torch.float32, dev, (nseq, Hv, dk, dv))
    f32 = dict(dtype=torch.float32, device=dev)
    gq, gk = torch.empty((B, T, Hqk, dk), **f32), torch.empty((B, T, Hqk, dk), **f32)
    gv = torch.empty((B, T, Hv, dv), **f32)
    gg, gb = torch.empty((B, T, Hv), **f32), torch.empty((B, T, Hv), **f32)
    gS0 = torch.empty((nseq, Hv, dk, dv), **f32) if want_grad_S0 else None
    gA = gdt = None
    with torch.cuda.device(dev):
        o, keep = _opts(lib, dt, scale, 64, normalize_qk, stream, dev, events)
        if cu_seqlens is not None:
            o.cu_seqlens = cu_seqlens.data_ptr()
            o.num_seqs = nseq
        if raw_gates is not None:
            A_log, dt_bias = raw_gates
            _need("A_log", A_log, torch.float32, dev, (Hv,))
            _need("dt_bias", dt_bias, torch.float32, dev, (Hv,))
            gA, gdt = torch.empty((Hv,), **f32), torch.empty((Hv,), **f32)
            o.flags |= L.GDN_RAW_GATES
            o.A_log, o.dt_bias = A_log.data_ptr(), dt_bias.data_ptr()
            o.grad_A_log, o.grad_dt_bias = gA.data_ptr(), gdt.data_ptr()
        need = int(lib.gdn_recurrent_bwd_workspace_size(B, T, Hqk, Hv, dk, dv, ctypes.byref(o)))
        if workspace is None:
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
        o.workspace = workspace.data_ptr()
        o.workspace_bytes = workspace.numel()
        st = lib.gdn_recurrent_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S0), _ptr(grad_out),
                                   _ptr(grad_S_final), _ptr(gq), _ptr(gk), _ptr(gv), _ptr(gg), _ptr(gb), _ptr(gS0),
                                   B, T, Hqk, Hv, dk, dv, ctypes.byref(o))
        del keep
        L.check(lib, st)
    if raw_gates is not None:
        return gq, gk, gv, gg, gb, gS0, gA, gdt
    return gq, gk, gv, gg, gb, gS0


def gdn_output_gate_fwd(o: torch.Tensor, z: torch.Tensor, norm_weight: torch.Tensor, eps: float = 1e-6, *,
                        out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """The shell's output gate on its own: o / sqrt(mean(o^2) + eps) * norm_weight * silu(z) over the last
    axis (dv of 32, 64 or 128).  o, z [..., dv] (bf16 or fp32, contiguous); out like o (may be o)."""
    lib = L.load()
    dev, dt = o.device, o.dtype
    if dt not in _DTYPES:
        raise ValueError(f"unsupported dtype {dt}")
    dv = int(o.shape[-1])
    _need("z", z, dt, dev, tuple(o.shape))
    _need("norm_weight", norm_weight, torch.float32, dev, (dv,))
    if not o.is_contiguous():
        raise ValueError("o must be contiguous")
    y = torch.empty_like(o) if out is None else out
    _need("out", y, dt, dev, tuple(o.shape))
    with torch.cuda.device(dev):
        op, keep = _opts(lib, dt, 1.0, 64, False, stream, dev, None)
        op.norm_eps = float(eps)
        st = lib.gdn_output_gate_fwd(_ptr(o), _ptr(z), _ptr(norm_weight), _ptr(y), o.numel() // dv, dv,
                                     ctypes.byref(op))
        del keep
        L.check(lib, st)
    return y


def gdn_output_gate_bwd(o: torch.Tensor, z: torch.Tensor, norm_weight: torch.Tensor, grad_y: torch.Tensor,
                        eps: float = 1e-6, *, stream: Optional[torch.cuda.Stream] = None):
    """Gradients through gdn_output_gate_fwd: returns fp32 (grad_o, grad_z like o, grad_norm_weight [dv])."""
    lib = L.load()
    dev, dt = o.device, o.dtype
    if dt not in _DTYPES:
        raise ValueError(f"unsupported dtype {dt}")
    dv = int(o.shape[-1])
    _need("z", z, dt, dev, tuple(o.shape))
    _need("grad_y", grad_y, dt, dev, tuple(o.shape))
    _need("norm_weight", norm_weight, torch.float32, dev, (dv,))
    rows = o.numel() // dv
    f32 = dict(dtype=torch.float32, device=dev)
    go, gz, gw = torch.empty(tuple(o.shape), **f32), torch.empty(tuple(o.shape), **f32), torch.empty((dv,), **f32)
    with torch.cuda.device(dev):
        op, keep = _opts(lib, dt, 1.0, 64, False, stream, dev, None)
        op.norm_eps = float(eps)
        need = int(lib.gdn_output_gate_bwd_workspace_size(rows, dv, ctypes.byref(op)))
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
        op.workspace, op.workspace_bytes = ws.data_ptr(), ws.numel()
        st = lib.gdn_output_gate_bwd(_ptr(o), _ptr(z), _ptr(norm_weight), _ptr(grad_y), _ptr(go), _ptr(gz),
                                     _ptr(gw), rows, dv, ctypes.byref(op))
        del keep
        L.check(lib, st)
    return go, gz, gw


def _token_rows(name, t, d, lead):
    """Elements between consecutive token rows of t ([*lead, heads, d] with contiguous heads, token rows evenly
    strided: a dense tensor or a slice of a packed projection).  Rows that share memory, a broadcast token's among them,
    are refused: the library takes a row stride of 0 for dense rows."""
    shape, stride = t.shape, t.stride()
    H = shape[lead]
    if lead == 1:
        row = stride[0] if shape[0] > 1 else H * d
        even = True
    else:
        row = stride[1] if shape[1] > 1 else stride[0] if shape[0] > 1 else H * d
        even = shape[0] <= 1 or stride[0] == shape[1] * row
    if even and row >= H * d and stride[lead + 1] == 1 and (H == 1 or stride[lead] == d):
        return row
    if t.numel():
        raise ValueError(f"{name} must have contiguous heads and evenly strided token rows of their own memory")
    return H * d


def _decay_inputs(q, k, v, log_decay, lead):
    """Shapes and row strides of the decayed attention's inputs (``lead`` leading dimensions)."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a tensor")
        if t.dim() != lead + 2:
            raise ValueError(f"{name} must be {lead + 2}-D [{'B, T' if lead == 2 else 'N'}, H, d]")
    dev, dt, qs, vs = q.device, q.dtype, q.shape, v.shape
    if dt not in _DTYPES:
        raise ValueError(f"unsupported dtype {dt}")
    if k.shape != qs:
        raise ValueError(f"k has shape {tuple(k.shape)}, expected {tuple(qs)}")
    if vs[0] != qs[0] or vs[lead - 1] != qs[lead - 1]:
        raise ValueError(f"v has shape {tuple(vs)}, expected leading {tuple(qs[:lead])}")
    if k.dtype is not dt or v.dtype is not dt or k.device != dev or v.device != dev:
        raise ValueError(f"q, k, v must have one type and device: {dt} on {dev}, {k.dtype} on {k.device}, "
                         f"{v.dtype} on {v.device}")
    Hqk, dk = qs[lead], qs[lead + 1]
    Hv, dv = vs[lead], vs[lead + 1]
    _need("log_decay", log_decay, torch.float32, dev, (Hv,))
    return dev, dt, Hqk, Hv, dk, dv, (_token_rows("q", q, dk, lead), _token_rows("k", k, dk, lead),
                                      _token_rows("v", v, dv, lead))


def _scratch(o, need, workspace, like):
    """Point the options at a workspace of at least ``need`` bytes (a new one: fp32 on the device of ``like``, an
    fp32 tensor); returns the tensor to keep alive."""
    if not need:
        return None
    if workspace is not None and (workspace.device != like.device or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on {like.device}")
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = like.new_empty((need + 3) // 4)
    o.workspace = workspace.data_ptr()
    o.workspace_bytes = workspace.numel() * workspace.element_size()
    return workspace


def _packed(o, cu_seqlens, B, dev):
    """Number of sequences; a packed call's offsets go into the options."""
    if cu_seqlens is None:
        return B
    if cu_seqlens.dim() != 1:
        raise ValueError("cu_seqlens must be 1-D")
    nseq = int(cu_seqlens.numel()) - 1
    _need("cu_seqlens", cu_seqlens, torch.int32, dev, (nseq + 1,))
    o.cu_seqlens = cu_seqlens.data_ptr()
    o.num_seqs = nseq
    return nseq


def gdn_decay_attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                       S0: Optional[torch.Tensor] = None, *, scale: float = 1.0,
                       cu_seqlens: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                       S_final: Optional[torch.Tensor] = None, output_final_state: bool = True,
                       workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None,
                       events: Optional[Sequence[int]] = None):
    """Linear attention with a decay for each value head, over whole sequences: S <- exp(log_decay[h]) S +
    k v^T, out = scale S^T q.  q, k [B, T, Hqk, dk]; v [B, T, Hv, dv] (bf16 or fp32; slices of a packed
    projection are taken as they are); log_decay fp32 [Hv] (<= 0); S0 [nseq, Hv, dk, dv] fp32 or None.  With
    ``cu_seqlens`` (int32 device tensor of nseq+1 offsets) B must be 1.  Returns (out [B, T, Hv, dv],
    S_final or None)."""
    lib = L.load()
    dev, dt, Hqk, Hv, dk, dv, strides = _decay_inputs(q, k, v, log_decay, 2)
    B, T = q.shape[:2]
    with _on(dev, stream):
        o, keep = _call_opts(lib, dt, scale, stream, dev, events)
        nseq = _packed(o, cu_seqlens, B, dev)
        if S0 is not None:
            _need("S0", S0, torch.float32, dev, (nseq, Hv, dk, dv))
        if out is None:
            out = torch.empty_like(v, memory_format=_DENSE)
        else:
            _need("out", out, dt, dev, (B, T, Hv, dv))
        if S_final is not None:
            _need("S_final", S_final, torch.float32, dev, (nseq, Hv, dk, dv))
        elif output_final_state:
            S_final = log_decay.new_empty((nseq, Hv, dk, dv)) if S0 is None else torch.empty_like(S0)
        workspace = _scratch(o, int(lib.gdn_decay_attn_fwd_workspace_size(B, T, Hqk, Hv, dk, dv, ctypes.byref(o))),
                             workspace, log_decay)
        st = lib.gdn_decay_attn_fwd(_ptr(q), strides[0], _ptr(k), strides[1], _ptr(v), strides[2], _ptr(log_decay),
                                    _ptr(S0), _ptr(out), _ptr(S_final), B, T, Hqk, Hv, dk, dv, ctypes.byref(o))
        del keep
        L.check(lib, st)
    return out, S_final


def gdn_decay_attn_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, S: torch.Tensor,
                        *, slots: Optional[torch.Tensor] = None, scale: float = 1.0,
                        out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None,
                        events: Optional[Sequence[int]] = None) -> torch.Tensor:
    """One token for each of N rows through gdn_decay_attn_fwd's recurrence.  q, k [N, Hqk, dk]; v [N, Hv, dv];
    S [pool, Hv, dk, dv] fp32, updated in place.  ``slots`` (int32 [N]) names each row's state in the pool
    (None: row n, state n); a row whose slot is outside the pool (-1, say) is idle and gets zeros.  Returns
    out [N, Hv, dv]."""
    lib = L.load()
    dev, dt, Hqk, Hv, dk, dv, strides = _decay_inputs(q, k, v, log_decay, 1)
    N = q.shape[0]
    pool = S.shape[0] if slots is not None and S.dim() == 4 else N
    _need("S", S, torch.float32, dev, (pool, Hv, dk, dv))
    if slots is not None:
        _need("slots", slots, torch.int32, dev, (N,))
    with _on(dev, stream):
        if out is None:
            out = torch.empty_like(v, memory_format=_DENSE)
        else:
            _need("out", out, dt, dev, (N, Hv, dv))
        o, keep = _call_opts(lib, dt, scale, stream, dev, events)
        st = lib.gdn_decay_attn_step(_ptr(q), strides[0], _ptr(k), strides[1], _ptr(v), strides[2], _ptr(log_decay),
                                     _ptr(S), _ptr(slots), pool, _ptr(out), N, Hqk, Hv, dk, dv, ctypes.byref(o))
        del keep
        L.check(lib, st)
    return out


def gdn_decay_attn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                       S0: Optional[torch.Tensor], grad_out: torch.Tensor,
                       grad_S_final: Optional[torch.Tensor] = None, *, scale: float = 1.0,
                       cu_seqlens: Optional[torch.Tensor] = None, want_grad_S0: bool = True,
                       grads: Optional[Sequence[torch.Tensor]] = None, workspace: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None, events: Optional[Sequence[int]] = None):
    """Gradients of a loss on (out, S_final) of gdn_decay_attn_fwd with respect to q, k, v and S0.  Inputs as
    there; grad_out like out (dense); grad_S_final fp32 like S_final or None.  ``grads`` = (grad_q, grad_k,
    grad_v) receives the three where given (slices of one packed tensor, say, as the convolution's backward
    takes them).  Returns (grad_q, grad_k, grad_v in the inputs' type, grad_S0 fp32 or None)."""
    lib = L.load()
    dev, dt, Hqk, Hv, dk, dv, strides = _decay_inputs(q, k, v, log_decay, 2)
    B, T = q.shape[:2]
    _need("grad_out", grad_out, dt, dev, (B, T, Hv, dv))
    with _on(dev, stream):
        if grads is None:
            grads = tuple(torch.empty_like(t, memory_format=_DENSE) for t in (q, k, v))
        else:
            for name, g, t in zip(("grad_q", "grad_k", "grad_v"), grads, (q, k, v)):
                if g.shape != t.shape or g.dtype != dt or g.device != dev:
                    raise ValueError(f"{name} must be {dt} of shape {tuple(t.shape)} on {dev}")
        gstrides = tuple(_token_rows(n, g, g.shape[3], 2) for n, g in zip(("grad_q", "grad_k", "grad_v"), grads))
        o, keep = _call_opts(lib, dt, scale, stream, dev, events)
        nseq = _packed(o, cu_seqlens, B, dev)
        for name, t in (("S0", S0), ("grad_S_final", grad_S_final)):
            if t is not None:
                _need(name, t, torch.float32, dev, (nseq, Hv, dk, dv))
        gS0 = log_decay.new_empty((nseq, Hv, dk, dv)) if want_grad_S0 else None
        workspace = _scratch(o, int(lib.gdn_decay_attn_bwd_workspace_size(B, T, Hqk, Hv, dk, dv, ctypes.byref(o))),
                             workspace, log_decay)
        st = lib.gdn_decay_attn_bwd(_ptr(q), strides[0], _ptr(k), strides[1], _ptr(v), strides[2], _ptr(log_decay),
                                    _ptr(S0), _ptr(grad_out), _ptr(grad_S_final), _ptr(grads[0]), gstrides[0],
                                    _ptr(grads[1]), gstrides[1], _ptr(grads[2]), gstrides[2], _ptr(gS0), B, T, Hqk, Hv,
                                    dk, dv, ctypes.byref(o))
        del keep
        L.check(lib, st)
    return grads[0], grads[1], grads[2], gS0


def _block_norm_inputs(x, b, post_weight, pre_weight, gate, res_scale):
    dev, dt = x.device, x.dtype
    if dt not in _DTYPES:
        raise ValueError(f"unsupported dtype {dt}")
    if x.dim() < 1:
        raise ValueError("x must be [..., D]")
    shape, D = tuple(x.shape), int(x.shape[-1])
    _need("x", x, dt, dev, shape)
    _need("b", b, dt, dev, shape)
    _need("post_weight", post_weight, torch.float32, dev, (D,))
    _need("pre_weight", pre_weight, torch.float32, dev, (D,))
    if res_scale is not None:
        _need("res_scale", res_scale, torch.float32, dev, (D,))
    if gate is not None:
        _need("gate", gate, dt, dev, shape if gate.shape[-1:] == x.shape[-1:] else shape[:-1] + (1,))
    return dev, dt, shape, D, (x.numel() // D if D else 0), (0 if gate is None else int(gate.shape[-1]))


def gdn_block_norm_fwd(x: torch.Tensor, b: torch.Tensor, post_weight: torch.Tensor, pre_weight: torch.Tensor, *,
                       gate: Optional[torch.Tensor] = None, res_scale: Optional[torch.Tensor] = None,
                       eps: float = 1e-6, out: Optional[Sequence[torch.Tensor]] = None,
                       stream: Optional[torch.cuda.Stream] = None, events: Optional[Sequence[int]] = None):
    """What surrounds a layer's block, in one pass: y = RMSNorm(b) post_weight, r = x + res_scale sigmoid(gate) y,
    n = RMSNorm(r) pre_weight.  x (residual stream) and b (the block's output) [..., D] (bf16 or fp32,
    contiguous); gate: logits like x, or [..., 1], or None (no gate); post_weight, pre_weight and res_scale
    (None: 1) fp32 [D].  ``out`` = (r, n) receives the results where given (r may be x, n may be b).
    Returns (r, n)."""
    lib = L.load()
    dev, dt, shape, D, rows, cols = _block_norm_inputs(x, b, post_weight, pre_weight, gate, res_scale)
    with _on(dev, stream):
        if out is None:
            r, n = torch.empty_like(x), torch.empty_like(x)
        else:
            r, n = out
            _need("r", r, dt, dev, shape)
            _need("n", n, dt, dev, shape)
        o, keep = _call_opts(lib, dt, 1.0, stream, dev, events)
        o.norm_eps = float(eps)
        st = lib.gdn_block_norm_fwd(_ptr(x), _ptr(b), _ptr(gate), cols, _ptr(res_scale), _ptr(post_weight),
                                    _ptr(pre_weight), _ptr(r), _ptr(n), rows, D, ctypes.byref(o))
        del keep
        L.check(lib, st)
    return r, n


def gdn_block_norm_bwd(x: torch.Tensor, b: torch.Tensor, post_weight: torch.Tensor, pre_weight: torch.Tensor,
                       grad_r: torch.Tensor, grad_n: torch.Tensor, *, gate: Optional[torch.Tensor] = None,
                       res_scale: Optional[torch.Tensor] = None, eps: float = 1e-6,
                       stream: Optional[torch.cuda.Stream] = None, events: Optional[Sequence[int]] = None):
    """Gradients through gdn_block_norm_fwd, from its inputs and grad_r, grad_n (like x).  Returns (grad_x,
    grad_b in x's type, grad_post_weight, grad_pre_weight fp32 [D], grad_gate like gate or None,
    grad_res_scale fp32 [D] or None)."""
    lib = L.load()
    dev, dt, shape, D, rows, cols = _block_norm_inputs(x, b, post_weight, pre_weight, gate, res_scale)
    _need("grad_r", grad_r, dt, dev, shape)
    _need("grad_n", grad_n, dt, dev, shape)
    with _on(dev, stream):
        gx, gb = torch.empty_like(x), torch.empty_like(x)
        gg = None if gate is None else torch.empty_like(gate)
        gpost, gpre = torch.empty_like(post_weight), torch.empty_like(post_weight)
        gs = None if res_scale is None else torch.empty_like(res_scale)
        o, keep = _call_opts(lib, dt, 1.0, stream, dev, events)
        o.norm_eps = float(eps)
        ws = _scratch(o, int(lib.gdn_block_norm_bwd_workspace_size(rows, D, ctypes.byref(o))), None, post_weight)
        st = lib.gdn_block_norm_bwd(_ptr(x), _ptr(b), _ptr(gate), cols, _ptr(res_scale), _ptr(post_weight),
                                    _ptr(pre_weight), _ptr(grad_r), _ptr(grad_n), _ptr(gx), _ptr(gb), _ptr(gg),
                                    _ptr(gpost), _ptr(gpre), _ptr(gs), rows, D, ctypes.byref(o))
        del keep, ws
        L.check(lib, st)
    return gx, gb, gpost, gpre, gg, gs


def _row_stride(name, t, lead, width):
    """Elements between consecutive token rows of t ([*lead, values] or [*lead, groups, values], contiguous behind
    ``lead``, ``width`` values in all): a dense tensor or a slice of a packed projection."""
    shape, stride = t.shape, t.stride()
    row = stride[lead - 1] if shape[lead - 1] > 1 else stride[0] if lead == 2 and shape[0] > 1 else width
    even = lead == 1 or shape[0] <= 1 or stride[0] == shape[1] * row
    inner = stride[-1] == 1 or shape[-1] == 1
    if len(shape) > lead + 1:
        inner = inner and (shape[lead] == 1 or stride[lead] == shape[lead + 1])
    if even and inner and row >= width:
        return row
    if t.numel():
        raise ValueError(f"{name} must have contiguous rows, evenly strided and of their own memory")
    return width


def _token_tensor(name, t, dt, dev, shape, lead, width):
    """Checks t and returns its row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype is not dt or t.shape != shape or t.device != dev:
        raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)} on {t.device}, expected {dt} {tuple(shape)} on {dev}")
    return width if t.is_contiguous() else _row_stride(name, t, lead, width)


def _scan_inputs(u, delta, A_log, B, C, skip, dt_bias, z, lead):
    """Sizes of the selective scan's inputs, and the arguments that its entry points begin with."""
    if not isinstance(u, torch.Tensor) or not isinstance(B, torch.Tensor) or not isinstance(A_log, torch.Tensor):
        raise TypeError("u, A_log and B must be tensors")
    us, bs, As = u.shape, B.shape, A_log.shape
    if len(us) != lead + 1 or len(bs) != lead + 2 or len(As) != 2:
        dims = "B, T" if lead == 2 else "N"
        raise ValueError(f"u must be [{dims}, D], B and C [{dims}, G, N], A_log [D, N]; they are {tuple(us)}, {tuple(bs)}, "
                         f"{tuple(As)}")
    dev, dt = u.device, u.dtype
    if dt not in _DTYPES:
        raise ValueError(f"unsupported dtype {dt}")
    D, G, N = us[lead], bs[lead], As[1]
    if bs[:lead] != us[:lead] or bs[lead + 1] != N:
        raise ValueError(f"B has shape {tuple(bs)}, expected {tuple(us[:lead]) + (G, N)}")
    _need("A_log", A_log, torch.float32, dev, (D, N))
    if skip is not None:
        _need("skip", skip, torch.float32, dev, (D,))
    if dt_bias is not None:
        _need("dt_bias", dt_bias, torch.float32, dev, (D,))
    GN = G * N
    return dev, dt, D, G, N, (
        u.data_ptr(), _token_tensor("u", u, dt, dev, us, lead, D),
        _pointer("delta", delta), _token_tensor("delta", delta, dt, dev, us, lead, D), A_log.data_ptr(),
        B.data_ptr(), _token_tensor("B", B, dt, dev, bs, lead, GN),
        _pointer("C", C), _token_tensor("C", C, dt, dev, bs, lead, GN), _ptr(skip), _ptr(dt_bias),
        None if z is None else _pointer("z", z), 0 if z is None else _token_tensor("z", z, dt, dev, us, lead, D))


def _pointer(name, t):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    return t.data_ptr()


def gdn_selective_scan_fwd(u: torch.Tensor, delta: torch.Tensor, A_log: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                           h0: Optional[torch.Tensor] = None, *, skip: Optional[torch.Tensor] = None,
                           dt_bias: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                           cu_seqlens: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                           h_final: Optional[torch.Tensor] = None, output_final_state: bool = True,
                           workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None,
                           events: Optional[Sequence[int]] = None):
    """The selective state space scan over whole sequences: dt = softplus(delta + dt_bias), h <- exp(-dt exp(A_log)) h +
    dt u B, y = (sum_n C h + skip u) silu(z).  u, delta and z (or None: no gate) [B, T, D], B and C [B, T, G, N] (bf16 or
    fp32; slices of packed projections are taken as they are); A_log fp32 [D, N] with N of 8, 16, 32 or 64; skip and
    dt_bias fp32 [D] or None (0); h0 [nseq, D, N] fp32 or None.  Channel d reads B and C of group d // (D // G).  With
    ``cu_seqlens`` (int32 device tensor of nseq+1 offsets) the batch must be 1.  ``out`` overlaps no input; ``h_final`` may be
    ``h0``.  Returns (y [B, T, D], h_final or None)."""
    lib = L.load()
    dev, dt, D, G, N, args = _scan_inputs(u, delta, A_log, B, C, skip, dt_bias, z, 2)
    nB, T = u.shape[:2]
    with _on(dev, stream):
        o, keep = _call_opts(lib, dt, 1.0, stream, dev, events)
        nseq = _packed(o, cu_seqlens, nB, dev)
        if h0 is not None:
            _need("h0", h0, torch.float32, dev, (nseq, D, N))
        if out is None:
            out = torch.empty_like(u, memory_format=_DENSE)
        else:
            _need("out", out, dt, dev, (nB, T, D))
        if h_final is not None:
            _need("h_final", h_final, torch.float32, dev, (nseq, D, N))
        elif output_final_state:
            h_final = A_log.new_empty((nseq, D, N)) if h0 is None else torch.empty_like(h0)
        workspace = _scratch(o, int(lib.gdn_selective_scan_fwd_workspace_size(nB, T, D, G, N, ctypes.byref(o))), workspace,
                             A_log)
        st = lib.gdn_selective_scan_fwd(*args, _ptr(h0), _ptr(out), _ptr(h_final), nB, T, D, G, N, ctypes.byref(o))
        del keep
        L.check(lib, st)
    return out, h_final


def gdn_selective_scan_step(u: torch.Tensor, delta: torch.Tensor, A_log: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                            h: torch.Tensor, *, skip: Optional[torch.Tensor] = None,
                            dt_bias: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                            slots: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                            stream: Optional[torch.cuda.Stream] = None,
                            events: Optional[Sequence[int]] = None) -> torch.Tensor:
    """One token for each of N rows through gdn_selective_scan_fwd's recurrence.  u, delta, z [N, D]; B, C [N, G, states];
    h [pool, D, states] fp32, updated in place.  ``slots`` (int32 [N]) names each row's state in the pool (None: row n,
    state n); a row whose slot is outside the pool (-1, say) is idle and gets zeros; ``out``
    overlaps no input.  Returns y [N, D]."""
    lib = L.load()
    dev, dt, D, G, N, args = _scan_inputs(u, delta, A_log, B, C, skip, dt_bias, z, 1)
    rows = u.shape[0]
    pool = h.shape[0] if slots is not None and h.dim() == 3 else rows
    _need("h", h, torch.float32, dev, (pool, D, N))
    if slots is not None:
        _need("slots", slots, torch.int32, dev, (rows,))
    with _on(dev, stream):
        if out is None:
            out = torch.empty_like(u, memory_format=_DENSE)
        else:
            _need("out", out, dt, dev, (rows, D))
        o, keep = _call_opts(lib, dt, 1.0, stream, dev, events)
        st = lib.gdn_selective_scan_step(*args, _ptr(h), _ptr(slots), pool, _ptr(out), rows, D, G, N, ctypes.byref(o))
        del keep
        L.check(lib, st)
    return out


def gdn_selective_scan_bwd(u: torch.Tensor, delta: torch.Tensor, A_log: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                           h0: Optional[torch.Tensor], grad_y: torch.Tensor, grad_h_final: Optional[torch.Tensor] = None,
                           *, skip: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None,
                           z: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
                           want_grad_h0: bool = True, grads: Optional[Sequence[torch.Tensor]] = None,
                           workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None,
                           events: Optional[Sequence[int]] = None):
    """Gradients of a loss on (y, h_final) of gdn_selective_scan_fwd.  Inputs as there; grad_y like y (dense);
    grad_h_final fp32 like h_final or None.  ``grads`` = (grad_B, grad_C, grad_z) receives those three where given
    (slices of packed gradients, say; grad_z None without z; none overlaps an input or another one).  The scratch, about
    D (N / 2 + N^2 / 128) bytes a token and 16 D N a sequence, is allocated where ``workspace`` is not large enough for it.
    Returns (grad_u, grad_delta in u's type, grad_A_log fp32, grad_B, grad_C in u's type, grad_skip, grad_dt_bias fp32 or
    None where the input is None, grad_z in u's type or None, grad_h0 fp32 or None)."""
    lib = L.load()
    dev, dt, D, G, N, args = _scan_inputs(u, delta, A_log, B, C, skip, dt_bias, z, 2)
    nB, T = u.shape[:2]
    _need("grad_y", grad_y, dt, dev, (nB, T, D))
    with _on(dev, stream):
        if grads is None:
            grads = (torch.empty_like(B, memory_format=_DENSE), torch.empty_like(C, memory_format=_DENSE),
                     None if z is None else torch.empty_like(z, memory_format=_DENSE))
        gB, gC, gz = grads
        if (gz is None) != (z is None):
            raise ValueError("grad_z goes with z")
        gb_stride = _token_tensor("grad_B", gB, dt, dev, B.shape, 2, G * N)
        gc_stride = _token_tensor("grad_C", gC, dt, dev, B.shape, 2, G * N)
        gz_stride = 0 if gz is None else _token_tensor("grad_z", gz, dt, dev, u.shape, 2, D)
        o, keep = _call_opts(lib, dt, 1.0, stream, dev, events)
        nseq = _packed(o, cu_seqlens, nB, dev)
        for name, t in (("h0", h0), ("grad_h_final", grad_h_final)):
            if t is not None:
                _need(name, t, torch.float32, dev, (nseq, D, N))
        gu, gd = torch.empty_like(u, memory_format=_DENSE), torch.empty_like(u, memory_format=_DENSE)
        gA = torch.empty_like(A_log)
        gs = None if skip is None else torch.empty_like(skip)
        gbias = None if dt_bias is None else torch.empty_like(dt_bias)
        gh0 = A_log.new_empty((nseq, D, N)) if want_grad_h0 else None
        workspace = _scratch(o, int(lib.gdn_selective_scan_bwd_workspace_size(nB, T, D, G, N, ctypes.byref(o))), workspace,
                             A_log)
        st = lib.gdn_selective_scan_bwd(*args, _ptr(h0), _ptr(grad_y), _ptr(grad_h_final), _ptr(gu), _ptr(gd), _ptr(gA),
                                        _ptr(gB), gb_stride, _ptr(gC), gc_stride, _ptr(gs), _ptr(gbias), _ptr(gz),
                                        gz_stride, _ptr(gh0), nB, T, D, G, N, ctypes.byref(o))
        del keep
        L.check(lib, st)
    return gu, gd, gA, gB, gC, gs, gbias, gz, gh0


def _layer_norm_inputs(x, weight, residual):
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a tensor")
    dev, dt = x.device, x.dtype
    if dt not in _DTYPES:
        raise ValueError(f"unsupported dtype {dt}")
    if x.dim() < 1:
        raise ValueError("x must be [..., D]")
    shape, D = x.shape, x.shape[-1]
    _need("x", x, dt, dev, shape)
    _need("weight", weight, torch.float32, dev, (D,))
    if residual is not None:
        _need("residual", residual, dt, dev, shape)
    return dev, dt, shape, D, (x.numel() // D if D else 0)


def gdn_layer_norm_fwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
                       residual: Optional[torch.Tensor] = None, eps: float = 1e-5,
                       out: Optional[Sequence[torch.Tensor]] = None, stream: Optional[torch.cuda.Stream] = None,
                       events: Optional[Sequence[int]] = None):
    """Layer norm with the residual add in front of it: r = x + residual (x where there is none), n = (r - mean(r)) /
    sqrt(var(r) + eps) weight + bias.  x and residual [..., D] (bf16 or fp32, contiguous); weight and bias (None: 0) fp32
    [D].  ``out`` = (n, r) receives the results where given (r None without a residual; each may be x or residual).
    Returns (n, r), r None without a residual."""
    lib = L.load()
    dev, dt, shape, D, rows = _layer_norm_inputs(x, weight, residual)
    if bias is not None:
        _need("bias", bias, torch.float32, dev, (D,))
    with _on(dev, stream):
        if out is None:
            n, r = torch.empty_like(x), None if residual is None else torch.empty_like(x)
        else:
            n, r = out
            _need("n", n, dt, dev, shape)
            if (r is None) != (residual is None):
                raise ValueError("r goes with residual")
            if r is not None:
                _need("r", r, dt, dev, shape)
        o, keep = _call_opts(lib, dt, 1.0, stream, dev, events)
        o.norm_eps = float(eps)
        st = lib.gdn_layer_norm_fwd(_ptr(x), _ptr(residual), _ptr(weight), _ptr(bias), _ptr(n), _ptr(r), rows, D,
                                    ctypes.byref(o))
        del keep
        L.check(lib, st)
    return n, r


def gdn_layer_norm_bwd(x: torch.Tensor, weight: torch.Tensor, grad_n: torch.Tensor, *,
                       residual: Optional[torch.Tensor] = None, grad_r: Optional[torch.Tensor] = None, eps: float = 1e-5,
                       want_grad_bias: bool = True, stream: Optional[torch.cuda.Stream] = None,
                       events: Optional[Sequence[int]] = None):
    """Gradients through gdn_layer_norm_fwd, from its inputs, grad_n and, for a residual stream that goes on, grad_r (like
    x).  Returns (grad_x in x's type, the gradient of x and of residual; grad_weight fp32 [D]; grad_bias fp32 [D] or
    None)."""
    lib = L.load()
    dev, dt, shape, D, rows = _layer_norm_inputs(x, weight, residual)
    _need("grad_n", grad_n, dt, dev, shape)
    if grad_r is not None:
        _need("grad_r", grad_r, dt, dev, shape)
    with _on(dev, stream):
        gx, gw = torch.empty_like(x), torch.empty_like(weight)
        gb = torch.empty_like(weight) if want_grad_bias else None
        o, keep = _call_opts(lib, dt, 1.0, stream, dev, events)
        o.norm_eps = float(eps)
        ws = _scratch(o, int(lib.gdn_layer_norm_bwd_workspace_size(rows, D, ctypes.byref(o))), None, weight)
        st = lib.gdn_layer_norm_bwd(_ptr(x), _ptr(residual), _ptr(weight), _ptr(grad_n), _ptr(grad_r), _ptr(gx), _ptr(gw),
                                    _ptr(gb), rows, D, ctypes.byref(o))
        del keep, ws
        L.check(lib, st)
    return gx, gw, gb
