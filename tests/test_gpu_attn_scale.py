"""Attention with scores of any size: scales up to the 2^64 that the entry
points take.  Queries and keys are small integers, so that every product is
exact; scales of 2^12 and more then leave no weight but those of the keys that
tie for the row's largest product, which are equal, whatever the scale's own
rounding is.  The bound is therefore the one of scores without an error (S =
0): the output's rounding, the weights' and the sums'."""
import pytest
import torch

import gated_deltanet_02_amd as G
from tests.attn_util import A, bound, check, cu_of, dtypes, f64, gen, make_pool, randn

pytestmark = pytest.mark.gpu
SCALES = [2.0 ** 12, 2.0 ** 19, -2.0 ** 24, 2.0 ** 28, -2.0 ** 33, 2.0 ** 35, 2.0 ** 60, -2.0 ** 64]


def i32(v):
    return torch.tensor(v, dtype=torch.int32)


def integers(g, *shape, dtype):
    x = torch.randint(-3, 4, shape, generator=g).to(dtype)
    x[1::7] = 0  # (rows that see all keys alike: the mean)
    return x


def check_rows(got, refs, dtype, label, step):
    at = 0
    for i, (out, M, S) in enumerate(refs):
        check(got[at: at + len(out)], out, bound(dtype, out, M, 0.0, step), f"{label} sequence {i}")
        at += len(out)


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("dtype", dtypes)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_decode_scales(d, dtype, scale):
    g, dt, lens = gen(d), dtypes[dtype], [700, 0, 1, 64, 33, 2500]
    k, v, table, _ = make_pool(g, lens, 16, 2, d, dt)
    k = integers(g, *k.shape, dtype=dt)
    q = integers(g, len(lens), 6, d, dtype=dt)
    got = G.gdn_attn_decode(q.cuda(), k.cuda(), v.cuda(), table.cuda(), i32(lens).cuda(), scale=scale)
    refs = [A.attention(f64(q[i: i + 1]), *(A.gather(f64(x), table[i].tolist(), n) for x in (k, v)), n - 1, scale=scale) for i, n in enumerate(lens)]
    check_rows(got, refs, dt, f"scale {scale}", True)


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("dtype", dtypes)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("lengths,H", [([300, 1, 0, 77], 4), ([520], 104)])  # keys shared between waves, and not
def test_prefill_scales(d, dtype, scale, paged, lengths, H):
    g, dt, Hk = gen(d + H), dtypes[dtype], 2
    starts = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
    T = starts[-1]
    q = integers(g, T, H, d, dtype=dt)
    if paged:
        k, v, table, _ = make_pool(g, lengths, 16, Hk, d, dt)
        k = integers(g, *k.shape, dtype=dt)
        rows = [[A.gather(f64(x), table[i].tolist(), n) for x in (k, v)] for i, n in enumerate(lengths)]
        how = dict(block_table=table.cuda(), seq_lens=i32(lengths).cuda())
    else:
        k, v = integers(g, T, Hk, d, dtype=dt), randn(g, T, Hk, d, dtype=dt)
        rows = [[f64(x[a:b]) for x in (k, v)] for a, b in zip(starts, starts[1:])]
        how = {}
    got = G.gdn_attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu_of(lengths).cuda(), scale=scale, **how)
    some = slice(0, H) if H < 16 else slice(0, H, 13)  # (heads checked: both key heads)
    kh = torch.arange(H)[some].numpy() // (H // Hk)
    refs = []
    for i, (a, b) in enumerate(zip(starts, starts[1:])):
        kr, vr = rows[i]
        refs.append(A.attention(f64(q[a:b, some]), kr[:, kh], vr[:, kh], 0, scale=scale))
    check_rows(got[:, some], refs, dt, f"scale {scale}", False)
