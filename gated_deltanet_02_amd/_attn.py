"""ctypes binding of the attention over a paged key-value cache
(include/gdn.h): block tables and slot maps, the store of new keys and values,
and the attention of prompts and of single tokens.

Argument marshalling only, as in ``_layer``.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional

import torch

from . import _binding as B
from ._layer import _describe, _like, _on


class GdnAttnOptions(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("window", ctypes.c_int32), ("sinks", ctypes.c_int32)]


_OPTIONS = struct.Struct("=fii")  # the same, packed
assert _OPTIONS.size == ctypes.sizeof(GdnAttnOptions)

_fns = None


def _functions():
    """The entry points of the loaded library, their prototypes set."""
    global _fns
    if _fns is None:
        L = B.lib()
        V, I = ctypes.c_void_p, ctypes.c_int32
        protos = {"gdn_cache_plan": [V] * 5 + [I] + [V] * 4,
                  "gdn_cache_release": [V] * 5 + [I, V],
                  "gdn_cache_store": [V] * 6,
                  "gdn_attn_prefill": [V] * 9,
                  "gdn_attn_decode": [V] * 8 + [ctypes.c_size_t, V],
                  "gdn_attn_workspace_size": [V, ctypes.POINTER(ctypes.c_size_t)]}
        for name, args in protos.items():
            f = getattr(L, name)
            f.argtypes, f.restype = args, ctypes.c_int
        L.gdn_attn_default_options.argtypes = [V]
        L.gdn_attn_default_options.restype = None
        _fns = L
    return _fns


def gdn_attn_default_options() -> GdnAttnOptions:
    o = GdnAttnOptions()
    _functions().gdn_attn_default_options(ctypes.addressof(o))
    return o


def _options(scale, window, sinks):
    """The packed options (0, as a float, is the C ABI's default scale and not
    a scale)."""
    if scale is not None and ctypes.c_float(scale).value == 0:
        raise ValueError("scale must not be 0 (None for 1 / sqrt(d))")
    buf = (ctypes.c_char * _OPTIONS.size)()
    _OPTIONS.pack_into(buf, 0, 0.0 if scale is None else scale, window, sinks)
    return buf


def _page_size(n):
    """A page size that its 32-bit argument holds (more bits would be cut)."""
    if not -1 << 31 <= n < 1 << 31:
        raise ValueError(f"page_size: more than 32 bits ({n})")
    return n


def gdn_cache_plan(ctx_lens, page_size: int, block_table, free_pages, n_free, cu_seqlens=None,
                   n_tokens: Optional[int] = None, seq_lens=None, slots=None, n_free_out=None, stream=None):
    """Block tables and slot maps from the requests' lengths: request i has
    ctx_lens[i] tokens in the cache and the new ones of ``cu_seqlens`` (one
    each without it), and takes the pages that these need off the stack
    free_pages[:n_free], in ``block_table`` [N, M] (in place), all of them or
    none.  ``n_tokens``: the packed batch's tokens (the size of ``slots``
    where that is not given).  Returns (seq_lens [N] int32, slots [T] int64,
    n_free_out [1] int32); seq_lens may be ctx_lens and n_free_out n_free.  A
    request that gets no pages keeps its length, its tokens' slots are -1 and
    their rows of the attention mean nothing: plan it again later."""
    L = _functions()
    page = _page_size(page_size)

    def body(device, handle):
        lens = torch.empty_like(ctx_lens) if seq_lens is None else seq_lens
        left = torch.empty_like(n_free) if n_free_out is None else n_free_out
        at = slots
        if at is None:
            if n_tokens is None and cu_seqlens is not None:
                raise ValueError("n_tokens or slots is required with cu_seqlens")
            n = ctx_lens.shape[0] if cu_seqlens is None else n_tokens
            at = torch.empty(n, dtype=torch.int64, device=device)
        keep, pc, pq, pt, pf, pn, pl, ps, po = _describe(device, (
            ("ctx_lens", ctx_lens), ("cu_seqlens", cu_seqlens), ("block_table", block_table),
            ("free_pages", free_pages), ("n_free", n_free), ("seq_lens", lens), ("slots", at),
            ("n_free_out", left)))
        B._check(L.gdn_cache_plan(pc, pq, pt, pf, pn, page, pl, ps, po, handle))
        return lens, at, left

    return _on(ctx_lens, stream, body)


def gdn_cache_release(done, seq_lens, page_size: int, block_table, free_pages, n_free, stream=None):
    """The pages of the requests with done[i] != 0 (int32) back onto the stack
    free_pages[:n_free] (entries below 0 are none); their lengths become 0.
    All but ``done`` in place."""
    L = _functions()
    page = _page_size(page_size)

    def body(device, handle):
        keep, pd, pl, pt, pf, pn = _describe(device, (
            ("done", done), ("seq_lens", seq_lens), ("block_table", block_table),
            ("free_pages", free_pages), ("n_free", n_free)))
        B._check(L.gdn_cache_release(pd, pl, pt, pf, pn, page, handle))

    return _on(done, stream, body)


def gdn_cache_store(k, v, slots, k_cache, v_cache, stream=None):
    """Rows of new keys and values [T, Hk, d] into their slots (int64 [T],
    those out of range are not stored) of the caches [pages, page_size, Hk,
    d]."""
    L = _functions()

    def body(device, handle):
        keep, pk, pv, ps, pkc, pvc = _describe(device, (
            ("k", k), ("v", v), ("slots", slots), ("k_cache", k_cache), ("v_cache", v_cache)))
        B._check(L.gdn_cache_store(pk, pv, ps, pkc, pvc, handle))

    return _on(k, stream, body)


def gdn_attn_prefill(q, k, v, cu_seqlens=None, block_table=None, seq_lens=None, scale: Optional[float] = None,
                     window: int = 0, sinks: int = 0, out=None, stream=None):
    """Causal attention of prompts: q [T, H, d] or [B, L, H, d], packed by
    ``cu_seqlens``; k, v [T, Hk, d], or with ``block_table`` [N, M] and
    ``seq_lens`` [N] (int32) the caches, of whose sequences the queries are
    the last tokens.  With a ``window`` a query sees that many keys, its own
    among them, and the first ``sinks``.  ``scale``: None for 1 / sqrt(d); 0
    is refused.
    Returns out."""
    L = _functions()
    o = _options(scale, window, sinks)

    def body(device, handle):
        y = _like(q) if out is None else out
        keep, pq, pk, pv, pc, pt, pl, po = _describe(device, (
            ("q", q), ("k", k), ("v", v), ("cu_seqlens", cu_seqlens), ("block_table", block_table),
            ("seq_lens", seq_lens), ("out", y)))
        B._check(L.gdn_attn_prefill(pq, pk, pv, pc, pt, pl, po, ctypes.addressof(o), handle))
        return y

    return _on(q, stream, body)


def gdn_attn_workspace_size(q) -> int:
    """Bytes of workspace that ``gdn_attn_decode`` needs (they follow q's dtype
    and d alone)."""
    L = _functions()
    keep, pq = _describe(q.device, (("q", q),))
    n = ctypes.c_size_t(0)
    B._check(L.gdn_attn_workspace_size(pq, ctypes.byref(n)))
    return n.value


def attn_workspace(q) -> torch.Tensor:
    """A device byte tensor large enough for ``gdn_attn_decode``."""
    return torch.empty(gdn_attn_workspace_size(q), dtype=torch.uint8, device=q.device)


def gdn_attn_decode(q, k_cache, v_cache, block_table, seq_lens, scale: Optional[float] = None, window: int = 0,
                    sinks: int = 0, out=None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of one new token for each of N sequences, the last of the
    seq_lens[i] (int32) that the caches [pages, page_size, Hk, d] hold through
    ``block_table`` [N, M] (int32): q [N, H, d].  ``window``, ``sinks`` and
    ``scale`` as ``gdn_attn_prefill``.  ``workspace``: a byte tensor from
    ``attn_workspace`` (allocated here if None).  Returns out [N, H, d]."""
    L = _functions()
    o = _options(scale, window, sinks)

    def body(device, handle):
        y, ws = _like(q) if out is None else out, workspace
        keep, pq, pk, pv, pt, pl, po, _ = _describe(device, (
            ("q", q), ("k_cache", k_cache), ("v_cache", v_cache), ("block_table", block_table),
            ("seq_lens", seq_lens), ("out", y), ("workspace", ws)))
        if ws is None:
            n = ctypes.c_size_t(0)
            B._check(L.gdn_attn_workspace_size(pq, ctypes.byref(n)))
            ws = torch.empty(n.value, dtype=torch.uint8, device=device)
        elif ws.dtype != torch.uint8 or not ws.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor")
        B._check(L.gdn_attn_decode(pq, pk, pv, pt, pl, po, ctypes.addressof(o), ws.data_ptr(), ws.numel(), handle))
        return y

    return _on(q, stream, body)
