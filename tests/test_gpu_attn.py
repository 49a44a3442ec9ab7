"""Attention of prompts and of single tokens over a paged cache against the
float64 reference, at the sizes, masks, strides and lengths where a kernel can
go wrong."""
import pytest
import torch

import gated_deltanet_02_amd as G
from tests.attn_util import A, bound, check, check_out, cu_of, dtypes, f64, gen, make_pool, randn, reference

pytestmark = pytest.mark.gpu
NAN = float("nan")


def i32(v):
    return torch.tensor(v, dtype=torch.int32)


# ---------------------------------------------------------------------------
# single tokens


def decode(seed, lens, H, Hk, d, dtype, page, window=0, sinks=0, scale=None, fill=NAN, width=None, label=""):
    g = gen(seed)
    k, v, table, _ = make_pool(g, lens, page, Hk, d, dtype, width=width, fill=fill)
    q = randn(g, len(lens), H, d, dtype=dtype)
    print(f"  decode {label} lens {lens[:8]} H {H} Hk {Hk} d {d} {dtype} page {page} window {window} sinks {sinks}", flush=True)
    got = G.gdn_attn_decode(q.cuda(), k.cuda(), v.cuda(), table.cuda(), i32(lens).cuda(), window=window, sinks=sinks, scale=scale)
    torch.cuda.synchronize()
    ref = reference(q, k, v, table, lens, list(range(len(lens) + 1)), window, sinks, scale)
    check_out(got, ref, dtype, label or "out", step=True)
    return got


@pytest.mark.parametrize("dtype", dtypes)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H,Hk", [(8, 8), (8, 2), (6, 1), (5, 5), (12, 4), (40, 2)])
def test_decode_heads(dtype, d, H, Hk):
    decode(d + H, [1, 100, 0, 33, 517], H, Hk, d, dtypes[dtype], 16)


@pytest.mark.parametrize("dtype", dtypes)
@pytest.mark.parametrize("page", [1, 7, 16, 48, 64, 1000])
def test_decode_pages(dtype, page):
    decode(page, [1, 15, 16, 17, 31, 32, 33, 0, 64, 65, 999, 1000, 1001, 2500], 4, 2, 64, dtypes[dtype], page)


@pytest.mark.parametrize("dtype", dtypes)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (33, 4), (100, 64), (100, 1), (5000, 3), (64, 5000), (0, 7)])
def test_decode_windows(dtype, window, sinks):
    lens = [0, 1, 2, 5, 15, 16, 17, 40, 99, 100, 101, 104, 164, 165, 1300]
    decode(window + sinks, lens, 4, 2, 128, dtypes[dtype], 24, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", dtypes)
def test_decode_many_short_and_one_long(dtype):
    lens = [(7 * i) % 61 for i in range(300)] + [20001] + [(5 * i) % 33 for i in range(100)]
    decode(5, lens, 4, 4, 64, dtypes[dtype], 16, fill=None)


def test_decode_all_empty():
    got = decode(6, [0, 0, 0], 4, 2, 128, torch.bfloat16, 16)
    assert (got == 0).all()


@pytest.mark.parametrize("scale", [0.01, 1.0, -0.3])
def test_decode_scale(scale):
    decode(7, [50, 700], 4, 2, 64, torch.float32, 16, scale=scale)


@pytest.mark.parametrize("dtype", dtypes)
def test_decode_large_scores(dtype):
    """Scores of hundreds: the maximum moves between tiles, weights underflow."""
    g = gen(8)
    dt, lens = dtypes[dtype], [700, 64]
    k, v, table, _ = make_pool(g, lens, 16, 2, 64, dt)
    q = (30 * randn(g, 2, 4, 64)).to(dt)
    got = G.gdn_attn_decode(q.cuda(), k.cuda(), v.cuda(), table.cuda(), i32(lens).cuda())
    check_out(got, reference(q, k, v, table, lens, [0, 1, 2]), dt, "large scores", step=True)


@pytest.mark.parametrize("dtype", dtypes)
def test_decode_strides(dtype):
    """Queries as a column range, head-major and interleaved caches, a table
    wider than it is used."""
    g, dt, lens, page, Hk, d = gen(9), dtypes[dtype], [77, 300, 5], 16, 2, 64
    k, v, table, _ = make_pool(g, lens, page, Hk, d, dt, width=40)
    rows = randn(g, 3, 10 * d, dtype=dt)
    q = rows[:, d: 5 * d].view(3, 4, d)
    ref = reference(q, k, v, table, lens, [0, 1, 2, 3])
    wide = torch.full((3, 60), -9, dtype=torch.int32)
    wide[:, 3:43] = table
    head_major = [x.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3) for x in (k, v)]
    both = torch.stack([k, v], 1).cuda()
    out = torch.zeros(3, 9 * d, dtype=dt, device="cuda")
    qg = rows.cuda()[:, d: 5 * d].view(3, 4, d)
    for name, (kc, vc) in {"head-major": head_major, "interleaved": (both[:, 0], both[:, 1])}.items():
        y = out[:, 2 * d: 6 * d].view(3, 4, d)
        G.gdn_attn_decode(qg, kc, vc, wide.cuda()[:, 3:43], i32(lens).cuda(), out=y)
        check_out(y, ref, dt, name, step=True)
    assert (out[:, : 2 * d] == 0).all() and (out[:, 6 * d:] == 0).all()


def test_decode_bad_pages_and_lengths():
    """Pages outside the cache hold nothing that is seen; lengths outside the
    table count as its ends."""
    g, lens, page = gen(10), [64, 64, 64, 64], 16
    k, v, table, _ = make_pool(g, lens, page, 2, 64, torch.float32, fill=NAN)
    q = randn(g, 4, 4, 64)
    bad = table.clone()
    bad[0, 1], bad[1, 3], bad[2, :] = -1, 10 ** 6, 2 ** 31 - 1
    got = G.gdn_attn_decode(q.cuda(), k.cuda(), v.cuda(), bad.cuda(), i32([64, 64, 64, 10 ** 9]).cuda())
    kd, vd = f64(k), f64(v)
    for i, keep in enumerate([list(range(16)) + list(range(32, 64)), list(range(48)), [], list(range(64))]):
        rows = [A.gather(x, table[i].tolist(), 64)[keep] for x in (kd, vd)]
        ref = A.attention(f64(q[i: i + 1]), *rows, len(keep) - 1)
        check_out(got[i: i + 1], ref, torch.float32, f"row {i}", step=True)
    got = G.gdn_attn_decode(q.cuda(), k.cuda(), v.cuda(), bad.cuda(), i32([-5] * 4).cuda())
    assert (got == 0).all()


def test_decode_one_sequence_over_the_chip():
    """A long sequence with one key head: every wave has a part."""
    decode(11, [70001], 3, 1, 64, torch.bfloat16, 64, fill=None)


def test_decode_repeats_bit_for_bit():
    g, lens = gen(12), [900, 13, 4000]
    k, v, table, _ = make_pool(g, lens, 16, 2, 128, torch.bfloat16)
    q = randn(g, 3, 8, 128, dtype=torch.bfloat16).cuda()
    args = (q, k.cuda(), v.cuda(), table.cuda(), i32(lens).cuda())
    ws = G.attn_workspace(q)
    first = G.gdn_attn_decode(*args, workspace=ws)
    for fill in (0, 255):
        ws.fill_(fill)
        assert torch.equal(G.gdn_attn_decode(*args, workspace=ws), first)


# ---------------------------------------------------------------------------
# prompts


def prefill(seed, lengths, H, Hk, d, dtype, window=0, sinks=0, scale=None, past=None, page=16, extra=0, cu=torch.int32):
    """Packed prompts, or with ``past`` chunks behind what the cache holds; the
    last ``extra`` rows are in no sequence."""
    g = gen(seed)
    T, starts = sum(lengths), [0]
    for n in lengths:
        starts.append(starts[-1] + n)
    q = randn(g, T + extra, H, d, dtype=dtype)
    out = torch.full((T + extra, H, d), 7.0, dtype=dtype, device="cuda")
    print(f"  prefill {lengths[:8]} past {past and past[:8]} H {H} Hk {Hk} d {d} {dtype} window {window} sinks {sinks}", flush=True)
    if past is None:
        k, v = (randn(g, T + extra, Hk, d, dtype=dtype) for _ in range(2))
        k[T:], v[T:] = NAN, NAN
        refs = [A.attention(f64(q[a:b]), f64(k[a:b]), f64(v[a:b]), 0, window, sinks, scale) for a, b in zip(starts, starts[1:])]
        G.gdn_attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu_of(lengths, cu).cuda(), window=window, sinks=sinks, scale=scale, out=out)
    else:
        lens = [a + b for a, b in zip(past, lengths)]
        k, v, table, _ = make_pool(g, lens, page, Hk, d, dtype, fill=NAN)
        refs = [A.attention(f64(q[a:b]), *(A.gather(f64(x), table[i].tolist(), lens[i]) for x in (k, v)), past[i], window, sinks, scale)
                for i, (a, b) in enumerate(zip(starts, starts[1:]))]
        G.gdn_attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu_of(lengths, cu).cuda(), block_table=table.cuda(), seq_lens=i32(lens).cuda(),
                           window=window, sinks=sinks, scale=scale, out=out)
    torch.cuda.synchronize()
    for i, ref in enumerate(refs):
        check_out(out[starts[i]: starts[i + 1]], ref, dtype, f"sequence {i} of {lengths[i]}")
    assert (out[T:] == 7).all(), "rows behind the last sequence changed"


EDGES = [1, 63, 0, 64, 65, 127, 128, 129, 31, 33, 257]


@pytest.mark.parametrize("dtype", dtypes)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H,Hk", [(4, 4), (6, 2), (3, 1)])
def test_prefill_heads(dtype, d, H, Hk):
    prefill(d + H, [100, 1, 0, 300], H, Hk, d, dtypes[dtype], extra=3)


@pytest.mark.parametrize("dtype", dtypes)
@pytest.mark.parametrize("cu", [torch.int32, torch.int64])
def test_prefill_lengths(dtype, cu):
    prefill(3, EDGES, 2, 1, 64, dtypes[dtype], extra=130, cu=cu)


@pytest.mark.parametrize("dtype", dtypes)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (33, 4), (64, 64), (100, 1), (100, 70), (5000, 3), (64, 5000), (0, 7), (200, 2)])
def test_prefill_windows(dtype, window, sinks):
    prefill(window + sinks, [600, 65, 1, 130], 2, 1, 128, dtypes[dtype], window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", dtypes)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [1, 16, 24, 64, 300])
def test_prefill_behind_a_cache(dtype, d, page):
    prefill(page, [5, 0, 64, 130, 1], 4, 2, d, dtypes[dtype], past=[0, 40, 300, 65, 511], page=page, extra=2)


@pytest.mark.parametrize("dtype", dtypes)
@pytest.mark.parametrize("window,sinks", [(1, 0), (33, 4), (100, 64), (300, 1)])
def test_prefill_behind_a_cache_with_windows(dtype, window, sinks):
    prefill(20, [5, 64, 130, 1], 4, 2, 64, dtypes[dtype], past=[0, 300, 65, 511], page=48, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", dtypes)
def test_prefill_uniform_batch(dtype):
    """[B, L, H, d] without cu_seqlens is B sequences."""
    g, dt = gen(30), dtypes[dtype]
    q, k, v = randn(g, 3, 150, 4, 64, dtype=dt), randn(g, 3, 150, 2, 64, dtype=dt), randn(g, 3, 150, 2, 64, dtype=dt)
    got = G.gdn_attn_prefill(q.cuda(), k.cuda(), v.cuda())
    for i in range(3):
        check_out(got[i], A.attention(f64(q[i]), f64(k[i]), f64(v[i]), 0), dt, f"sequence {i}")


@pytest.mark.parametrize("dtype", dtypes)
def test_prefill_strides(dtype):
    """q, k and v as column ranges of one array, out as one of another."""
    g, dt, T, H, Hk, d = gen(31), dtypes[dtype], 333, 4, 2, 128
    rows = randn(g, T, (H + 2 * Hk) * d, dtype=dt).cuda()
    q, k, v = rows[:, : H * d].view(T, H, d), rows[:, H * d: (H + Hk) * d].view(T, Hk, d), rows[:, (H + Hk) * d:].view(T, Hk, d)
    out = torch.zeros(T, (H + 2) * d, dtype=dt, device="cuda")
    G.gdn_attn_prefill(q, k, v, out=out[:, d: (H + 1) * d].view(T, H, d))
    check_out(out[:, d: (H + 1) * d].view(T, H, d), A.attention(f64(q), f64(k), f64(v), 0), dt, "column ranges")
    assert (out[:, :d] == 0).all() and (out[:, (H + 1) * d:] == 0).all()


@pytest.mark.parametrize("dtype", dtypes)
def test_prefill_large_scores(dtype):
    g, dt = gen(32), dtypes[dtype]
    q, k, v = (30 * randn(g, 300, 2, 64)).to(dt), randn(g, 300, 2, 64, dtype=dt), randn(g, 300, 2, 64, dtype=dt)
    got = G.gdn_attn_prefill(q.cuda(), k.cuda(), v.cuda())
    check_out(got, A.attention(f64(q), f64(k), f64(v), 0), dt, "large scores")


def test_prefill_more_new_tokens_than_the_cache_holds():
    """Queries before a sequence's first token see nothing."""
    g = gen(33)
    k, v, table, _ = make_pool(g, [20], 16, 2, 64, torch.float32, fill=NAN)
    q = randn(g, 50, 2, 64)
    got = G.gdn_attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu_of([50]).cuda(), block_table=table.cuda(), seq_lens=i32([20]).cuda())
    rows = [A.gather(f64(x), table[0].tolist(), 20) for x in (k, v)]
    check_out(got, A.attention(f64(q), *rows, -30), torch.float32, "30 rows before the first token")
    assert (got[:30] == 0).all()


def test_prefill_bad_pages():
    g = gen(34)
    k, v, table, _ = make_pool(g, [100], 16, 1, 64, torch.bfloat16, fill=NAN)
    q = randn(g, 100, 1, 64, dtype=torch.bfloat16)
    bad = table.clone()
    bad[0, 2], bad[0, 4] = -3, 10 ** 8
    got = G.gdn_attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu_of([100]).cuda(), block_table=bad.cuda(), seq_lens=i32([100]).cuda())
    keep = [j for j in range(100) if j // 16 not in (2, 4)]
    kd, vd = (A.gather(f64(x), table[0].tolist(), 100)[keep] for x in (k, v))
    for p in (0, 31, 32, 47, 48, 70, 99):
        n = sum(j <= p for j in keep)
        check_out(got[p: p + 1], A.attention(f64(q[p: p + 1]), kd[:n], vd[:n], n - 1), torch.bfloat16, f"row {p}")


def test_prefill_malformed_starts_stay_in_range():
    g = gen(35)
    q, k, v = (randn(g, 200, 2, 64, dtype=torch.bfloat16).cuda() for _ in range(3))
    for cu in ([0, 150, 100, 200], [5, 5000, 10 ** 9, 3], [-4, 0, 0, 200]):
        out = G.gdn_attn_prefill(q, k, v, i32(cu).cuda())
        torch.cuda.synchronize()
        assert out.shape == q.shape


def test_prefill_a_step_at_a_time_is_decode():
    """A prompt in chunks, then single tokens: the rows of the whole prompt."""
    g, T, H, Hk, d, page = gen(36), 200, 4, 2, 64, 16
    q, k, v = randn(g, T, H, d), randn(g, T, Hk, d), randn(g, T, Hk, d)
    whole = G.gdn_attn_prefill(q.cuda(), k.cuda(), v.cuda())
    table = torch.randperm(13, generator=g).to(torch.int32).view(1, 13).cuda()
    slots = (table[0].long()[torch.arange(T) // page] * page + torch.arange(T).cuda() % page)
    kc, vc = (torch.full((13, page, Hk, d), NAN, device="cuda") for _ in range(2))
    ref = A.attention(f64(q), f64(k), f64(v), 0)
    for a, b in ((0, 70), (70, 71), (71, 190)):
        G.gdn_cache_store(k[a:b].cuda(), v[a:b].cuda(), slots[a:b].contiguous(), kc, vc)
        out = G.gdn_attn_prefill(q[a:b].cuda(), kc, vc, cu_of([b - a]).cuda(), block_table=table, seq_lens=i32([b]).cuda())
        check(out, ref[0][a:b], bound(torch.float32, *(x[a:b] for x in ref), False), f"chunk {a}:{b}")
    for t in range(190, 200):
        G.gdn_cache_store(k[t:t + 1].cuda(), v[t:t + 1].cuda(), slots[t:t + 1].contiguous(), kc, vc)
        out = G.gdn_attn_decode(q[t:t + 1].cuda(), kc, vc, table, i32([t + 1]).cuda())
        check(out, ref[0][t:t + 1], bound(torch.float32, *(x[t:t + 1] for x in ref), True), f"token {t}")
    check_out(whole, ref, torch.float32, "whole")


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 64), (torch.bfloat16, 128), (torch.bfloat16, 256), (torch.float32, 128)])
@pytest.mark.parametrize("scale", [0.02, -0.2])
def test_prefill_scale(dtype, d, scale):
    prefill(70, [300, 1, 77], 4, 2, d, dtype, scale=scale)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lengths,H", [([300], 128), ([4000], 16), ([4225], 16), ([200, 0, 3300, 9], 20)])
def test_prefill_around_the_split(d, lengths, H):
    """Few and many (tile, head) pairs: keys shared by two groups of waves, or not."""
    prefill(71, lengths, H, 2, d, torch.bfloat16)


@pytest.mark.parametrize("lengths", [[8193], [2048, 17, 900]])
def test_prefill_window_around_the_split(lengths):
    prefill(72, lengths, 4, 2, 128, torch.bfloat16, window=130, sinks=70)


@pytest.mark.parametrize("d,dtype", [(64, torch.bfloat16), (128, torch.bfloat16), (256, torch.bfloat16), (128, torch.float32)])
@pytest.mark.parametrize("n", [1, 3, 16, 40, 200])
def test_decode_one_long_among_short(d, dtype, n):
    """Chains of one part, of a few and of hundreds, joined by one wave or by all."""
    lens = [3 + 7 * i % 90 for i in range(n)]
    lens[n // 2] = 30000
    decode(73, lens, 6, 2, d, dtype, 16)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lengths,H", [([700], 4), ([17, 0, 16, 300, 15], 6), ([2049], 8), ([1700], 10)])
@pytest.mark.parametrize("past", [False, True])
def test_prefill_f32_around_the_split(d, lengths, H, past):
    """Few and many workgroups: keys shared out among the waves, or queries."""
    prefill(74, lengths, H, 2, d, torch.float32, past=[5 + 41 * i for i in range(len(lengths))] if past else None)
