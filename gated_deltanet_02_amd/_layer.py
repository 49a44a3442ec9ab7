"""ctypes binding of the operators around a recurrent layer's projections
(include/gdn.h): the short convolution, the selective state space scan and
step, and the residual norm.

Argument marshalling only, as in ``_binding``: tensors become ``gdn_tensor``
descriptors, the current HIP stream of the tensors' device is passed through,
and a bad status raises ``GdnError``.  What a call allocates itself (an
output that was not given, a workspace) comes from the pool of the stream
that the kernels run on.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional

import torch

from . import _binding as B

SSM_SOFTPLUS = 1
CONV_SILU = 1
E4M3 = 5

_CODES = {torch.bfloat16: 1, torch.float32: 2, torch.int32: 3, torch.int64: 4,
          torch.float8_e4m3fn: E4M3}
# gdn_tensor by rank: data, dtype, ndim, shape[4], stride[4]
_DESC = {n: struct.Struct(f"=Qii{n}q{8 * (4 - n)}x{n}q{8 * (4 - n)}x") for n in range(1, 5)}
_DESC_BYTES = ctypes.sizeof(B.GdnTensor)
assert all(s.size == _DESC_BYTES for s in _DESC.values())


class GdnSsmOptions(ctypes.Structure):
    _fields_ = [("a_log", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p),
                ("d_skip", ctypes.c_void_p), ("flags", ctypes.c_uint32),
                ("segment_blocks", ctypes.c_int32)]


_OPTIONS = struct.Struct("=QQQIi")  # the same, packed
assert _OPTIONS.size == ctypes.sizeof(GdnSsmOptions)


_fns = None


def _functions():
    """The entry points of the loaded library, their prototypes set."""
    global _fns
    if _fns is None:
        L = B.lib()
        V = ctypes.c_void_p
        protos = {"gdn_short_conv": [V] * 7 + [ctypes.c_uint32, V],
                  "gdn_ssm_prefill": [V] * 10 + [ctypes.c_size_t, V],
                  "gdn_ssm_workspace_size": [V] * 4 + [ctypes.POINTER(ctypes.c_size_t)],
                  "gdn_ssm_decode": [V] * 8,
                  "gdn_add_rms_norm": [V] * 3 + [ctypes.c_float] + [V] * 5}
        for name, args in protos.items():
            f = getattr(L, name)
            f.argtypes, f.restype = args, ctypes.c_int
        L.gdn_ssm_default_options.argtypes = [V]
        L.gdn_ssm_default_options.restype = None
        _fns = L
    return _fns


def _describe(device, named):
    """Descriptors of the named tensors in one buffer (kept by the caller
    while it is used; room for the scan's options at its end), and the
    address of each (None for None).  All tensors must be on ``device``."""
    buf = (ctypes.c_char * (_DESC_BYTES * len(named) + _OPTIONS.size))()
    base = ctypes.addressof(buf)
    index = device.index
    at = [buf]
    for name, t in named:
        if t is None:
            at.append(None)
            continue
        if t.get_device() != index:
            raise ValueError(f"{name} must be a GPU tensor on {device} (got {t.device})")
        shape = t.shape
        n = len(shape)
        if not 1 <= n <= 4:
            raise ValueError(f"{name}: 1 to 4 dimensions")
        off = (len(at) - 1) * _DESC_BYTES
        _DESC[n].pack_into(buf, off, t.data_ptr(), _CODES.get(t.dtype, 0), n, *shape, *t.stride())
        at.append(base + off)
    return at


def _vector(t: Optional[torch.Tensor], name: str, n: int, device):
    """Address of an f32 vector of n values (None -> NULL)."""
    if t is None:
        return None
    if t.dtype != torch.float32 or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of {n} values")
    if t.get_device() != device.index:
        raise ValueError(f"{name} must be a GPU tensor on {device} (got {t.device})")
    return t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on(x, stream, body):
    """body(device, stream handle), with ``stream`` (default: the current
    one of x's device) current: allocations and launches belong to it."""
    device = x.device
    if device.type != "cuda":
        raise ValueError(f"x must be a GPU tensor (got {device})")
    if stream is not None:
        s = B._torch_stream(stream, device)
        with torch.cuda.stream(s):
            return body(device, s.cuda_stream)
    if _current_device() == device.index:  # (x is on a GPU: torch has initialised it)
        return body(device, _raw_stream(device.index))
    with torch.cuda.device(device):
        return body(device, _raw_stream(device.index))


def _like(x):
    if x.is_contiguous():
        return torch.empty_like(x)
    return torch.empty(x.shape, dtype=x.dtype, device=x.device)


def gdn_ssm_default_options() -> GdnSsmOptions:
    o = GdnSsmOptions()
    _functions().gdn_ssm_default_options(ctypes.addressof(o))
    return o


def gdn_short_conv(x, weight, bias=None, cu_seqlens=None, state_in=None, state_out=None,
                   silu: bool = False, out=None, stream=None):
    """The causal depthwise convolution along each sequence's tokens, with
    an optional silu.  x [T, D] (one sequence, or packed by ``cu_seqlens``)
    or [B, L, D] (L = 1: one step of B running sequences); weight f32 [D, W],
    W = 1 .. 4, the last tap on the current token; bias f32 [D];
    ``state_in`` / ``state_out`` [N, W - 1, D] the rows before each sequence
    (None: zeros) and its last rows (None: not written; may be
    ``state_in``).  Returns out."""
    L = _functions()

    def body(device, handle):
        y = _like(x) if out is None else out
        keep, px, pw, pc, pi, ps, po = _describe(device, (
            ("x", x), ("weight", weight), ("cu_seqlens", cu_seqlens), ("state_in", state_in),
            ("state_out", state_out), ("out", y)))
        pb = _vector(bias, "bias", x.shape[-1], device)
        B._check(L.gdn_short_conv(px, pw, pb, pc, pi, ps, po, CONV_SILU if silu else 0, handle))
        return y

    return _on(x, stream, body)


def _ssm_options(keep, a_log, dt_bias, d_skip, softplus, segment_blocks, x, device):
    """Packs the options behind the descriptors in ``keep``; their address."""
    heads = x.shape[-2] if x.dim() > 1 else 0
    off = len(keep) - _OPTIONS.size
    _OPTIONS.pack_into(keep, off, _vector(a_log, "a_log", heads, device) or 0,
                       _vector(dt_bias, "dt_bias", heads, device) or 0, _vector(d_skip, "d_skip", heads, device) or 0,
                       SSM_SOFTPLUS if softplus else 0, segment_blocks)
    return ctypes.addressof(keep) + off


def gdn_ssm_workspace_size(x, b, cu_seqlens=None, segment_blocks: int = 0) -> int:
    """Bytes of workspace that ``gdn_ssm_prefill`` needs for these shapes."""
    L = _functions()
    o = GdnSsmOptions()
    o.flags, o.segment_blocks = SSM_SOFTPLUS, segment_blocks
    keep, px, pb, pc = _describe(x.device, (("x", x), ("b", b), ("cu_seqlens", cu_seqlens)))
    n = ctypes.c_size_t(0)
    B._check(L.gdn_ssm_workspace_size(px, pb, pc, ctypes.addressof(o), ctypes.byref(n)))
    return n.value


def ssm_workspace(x, b, cu_seqlens=None, segment_blocks: int = 0) -> torch.Tensor:
    """A device byte tensor large enough for ``gdn_ssm_prefill``."""
    n = gdn_ssm_workspace_size(x, b, cu_seqlens, segment_blocks)
    return torch.empty(max(n, 1), dtype=torch.uint8, device=x.device)


def gdn_ssm_prefill(x, dt, b, c, a_log=None, dt_bias=None, d_skip=None, cu_seqlens=None,
                    init_state=None, out=None, final_state=None, softplus: bool = True,
                    segment_blocks: int = 0, workspace: Optional[torch.Tensor] = None, stream=None):
    """The selective state space scan over prompts: for each sequence and
    head, S <- exp(-exp(a_log) d) S + d b x^T and out = S^T c + d_skip x, with
    d = softplus(dt + dt_bias) (``softplus=False``: d = dt + dt_bias, >= 0).
    x [T, H, P] or [B, L, H, P]; dt f32 [T, H]; b, c [T, G, N] (head h reads
    group h / (H/G)); states f32 [N_seq, H, N, P], ``final_state`` written
    only when given (it may be ``init_state``).  ``workspace``: a byte tensor
    from ``ssm_workspace`` (allocated here if None).  Returns
    (out, final_state)."""
    L = _functions()

    def body(device, handle):
        y, ws = _like(x) if out is None else out, workspace
        keep, px, pd, pb, pc, pq, pi, po, pf, _ = _describe(device, (
            ("x", x), ("dt", dt), ("b", b), ("c", c), ("cu_seqlens", cu_seqlens),
            ("init_state", init_state), ("out", y), ("final_state", final_state),
            ("workspace", ws)))
        at = _ssm_options(keep, a_log, dt_bias, d_skip, softplus, segment_blocks, x, device)
        if ws is None:
            n = ctypes.c_size_t(0)
            B._check(L.gdn_ssm_workspace_size(px, pb, pq, at, ctypes.byref(n)))
            if n.value:
                ws = torch.empty(n.value, dtype=torch.uint8, device=device)
        elif ws.dtype != torch.uint8 or not ws.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor")
        where, size = (ws.data_ptr(), ws.numel()) if ws is not None else (None, 0)
        B._check(L.gdn_ssm_prefill(px, pd, pb, pc, pq, pi, po, pf, at, where, size, handle))
        return y, final_state

    return _on(x, stream, body)


def gdn_ssm_decode(x, dt, b, c, state, a_log=None, dt_bias=None, d_skip=None, out=None,
                   softplus: bool = True, stream=None):
    """One token of the scan for each of N running sequences: ``state`` f32
    [N, H, n, p] is updated in place.  x [N, H, p]; dt f32 [N, H]; b, c
    [N, G, n].  Returns out [N, H, p]."""
    L = _functions()

    def body(device, handle):
        y = _like(x) if out is None else out
        keep, px, pd, pb, pc, ps, po = _describe(device, (
            ("x", x), ("dt", dt), ("b", b), ("c", c), ("state", state), ("out", y)))
        at = _ssm_options(keep, a_log, dt_bias, d_skip, softplus, 0, x, device)
        B._check(L.gdn_ssm_decode(px, pd, pb, pc, ps, po, at, handle))
        return y

    return _on(x, stream, body)


def gdn_add_rms_norm(x, residual=None, weight=None, eps: float = 1e-6, residual_out=None, out=None,
                     out_q=None, scales=None, stream=None):
    """r = x + residual and y = r / sqrt(mean(r^2) + eps) * weight over the
    rows of x [R, D], into those of residual_out (r), out (y) and out_q with
    scales (y in float8_e4m3fn; scales f32 [R], or [R, ceil(D / 128)] for a
    scale per 128 columns) that are given; ``out`` is allocated if neither it
    nor ``out_q`` is.  residual_out and out may be x or residual.  Returns
    (out, residual_out, out_q, scales)."""
    L = _functions()

    def body(device, handle):
        y = _like(x) if out is None and out_q is None else out
        keep, px, pr, pro, po, pq, ps = _describe(device, (
            ("x", x), ("residual", residual), ("residual_out", residual_out), ("out", y),
            ("out_q", out_q), ("scales", scales)))
        pw = _vector(weight, "weight", x.shape[-1], device)
        B._check(L.gdn_add_rms_norm(px, pr, pw, eps, pro, po, pq, ps, handle))
        return y, residual_out, out_q, scales

    return _on(x, stream, body)
