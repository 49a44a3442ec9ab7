"""A NaN or infinity among the keys or values of a prompt: in a key it reaches
the rows that see it, in a value at most the tiles of 128 queries that hold one
of these.  All other rows are what they are without it."""
import numpy as np
import pytest
import torch

import gated_deltanet_02_amd as G
from tests.attn_util import A, bound, check, cu_of, dtypes, f64, gen, make_pool, randn

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32)


@pytest.mark.parametrize("dtype", dtypes)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 0), (150, 3)])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("H", [2, 128])  # keys shared between waves, and not
def test_what_a_nan_reaches(dtype, d, window, sinks, paged, H):
    g, dt, Hk = gen(d + window), dtypes[dtype], 2
    lengths, bad = [700, 300], [1, 200, 455]  # places in the first sequence
    T = sum(lengths)
    q = randn(g, T, H, d, dtype=dt)
    if paged:
        k0, v0, table, _ = make_pool(g, lengths, 16, Hk, d, dt, fill=float("nan"))
        at = [(int(table[0, p // 16]), p % 16) for p in range(lengths[0])]
        how = dict(block_table=table.cuda(), seq_lens=i32(lengths).cuda())
        rows = [[A.gather(f64(x), table[i].tolist(), n) for x in (k0, v0)] for i, n in enumerate(lengths)]
    else:
        k0, v0 = randn(g, T, Hk, d, dtype=dt), randn(g, T, Hk, d, dtype=dt)
        at = [(p,) for p in range(lengths[0])]
        how = {}
        rows = [[f64(x[a:b]) for x in (k0, v0)] for a, b in ((0, 700), (700, 1000))]
    some = [0, H - 1]
    refs = [A.attention(f64(q[a:b, some]), *rows[i], 0, window, sinks) for i, (a, b) in enumerate(((0, 700), (700, 1000)))]
    out, M, S = (np.concatenate([r[i] for r in refs]) for i in range(3))
    see = np.stack([A.seen(p, 700, window, sinks) for p in range(700)])[:, bad].any(1)
    tiles = np.repeat([see[i: i + 128].any() for i in range(0, 700, 128)], 128)[:700]
    for kind in ("key", "value"):
        for what in (float("nan"), float("inf")):
            k, v = k0.clone(), v0.clone()
            for p in bad:
                (k if kind == "key" else v)[at[p]] = what
            got = f64(G.gdn_attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu_of(lengths).cuda(), window=window, sinks=sinks, **how))[:, some]
            reached = np.concatenate([see if kind == "key" else tiles, np.zeros(300, bool)])
            check(got[~reached], out[~reached], bound(dt, out, M, S, False)[~reached], f"{kind} {what}")
            if kind == "value" or what != what:
                assert not np.isfinite(got[:700][see]).any(), f"{kind} {what}: rows that see it"
