"""Inputs, derived tolerances and checks of the tests of the attention over a
paged cache (not collected by pytest).

Tolerances.  A rounding to a type costs at most half a step, ``HALF[dtype]``
relative to the value.  Let M be the sum of a row's weights times |v|, and S
the largest sum of |q k| of a key it sees, times the scale.  A score is a sum
of at most 256 fp32 products; MFMA adds them in short chains, so it is off by
less than 2^-18 S (64 roundings' worth), which multiplies its weight by as
much; the weights' exponentials, their running maximum's rescaling and the
sums of up to some 2^14 terms in fp32, tree-like in the main, cost less than
2^-17 more: together 2^-16 (1 + S) M.  bf16 weights of prompts add half a step
each, 2^-8 M at most; those of single tokens enter as two terms, 2^-16 M
(within the same bound as the rest, counted as 2^-15 (1 + S) M).
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import attention as A
from tests.layer_util import HALF, check, cu_of, f64, gen, randn

__all__ = ["A", "HALF", "bound", "check", "check_out", "cu_of", "f64", "gen", "make_pool", "randn", "dtypes"]

dtypes = {"bf16": torch.bfloat16, "f32": torch.float32}


def bound(dtype, out, M, S, step):
    if dtype == torch.bfloat16:
        return HALF[dtype] * np.abs(out) + ((2.0 ** -15 if step else 2.0 ** -16) * (1 + S) + (0 if step else 2.0 ** -8)) * M
    return HALF[dtype] * np.abs(out) + 2.0 ** -16 * (1 + S) * M


def check_out(got, ref, dtype, label, step=False):
    out, M, S = ref
    # (a row that sees nothing is exactly zero)
    check(got, out, bound(dtype, out, M, S, step) + (M == 0) * 0.0, label)


def make_pool(g, lens, page, Hk, d, dtype, spare=3, width=None, fill=None):
    """Caches on the CPU with pages in no order; the places behind a
    sequence's end and the pages of nobody hold ``fill`` (NaN, say)."""
    have = [-(-n // page) for n in lens]
    pages = sum(have) + spare
    order = torch.randperm(pages, generator=g).to(torch.int32)
    M = width if width is not None else max([1] + have)
    table = torch.full((len(lens), M), -7, dtype=torch.int32)
    at = 0
    for i, n in enumerate(have):
        table[i, :n] = order[at: at + n]
        at += n
    k, v = (randn(g, pages, page, Hk, d, dtype=dtype) for _ in range(2))
    if fill is not None:
        live = torch.zeros(pages, page, dtype=torch.bool)
        for i, n in enumerate(lens):
            for p in range(n):
                live[table[i, p // page], p % page] = True
        k[~live] = fill
        v[~live] = fill
    return k, v, table, order[at:]


def reference(q, kc, vc, table, lens, starts, window=0, sinks=0, scale=None):
    """The rows of all sequences from the caches: (out, M, S)."""
    parts = []
    kc, vc = f64(kc), f64(vc)
    for i, n in enumerate(lens):
        a, b = int(starts[i]), int(starts[i + 1])
        k, v = A.gather(kc, table[i].tolist(), n), A.gather(vc, table[i].tolist(), n)
        parts.append(A.attention(f64(q[a:b]), k, v, n - (b - a), window, sinks, scale))
    return tuple(np.concatenate([p[i] for p in parts]) for i in range(3))
