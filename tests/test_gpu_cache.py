"""Block tables and slot maps, the release of pages and the store of rows
against serial references: whole numbers and copies, equal bit for bit."""
import numpy as np
import pytest
import torch

import gated_deltanet_02_amd as G
from tests.attn_util import A, cu_of, dtypes, gen, randn

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32)


def tables(rng, ctx, width, page, spare):
    have = [min(-(-c // page), width) for c in ctx]
    order = rng.permutation(sum(have) + spare).astype(np.int32)
    table, at = np.full((len(ctx), width), -1, np.int32), 0
    for i, n in enumerate(have):
        table[i, :n] = order[at: at + n]
        at += n
    return table, order[at:]


def run_plan(ctx, new, table, free, n_free, page, extra=0, cu=torch.int32, in_place=False, wide=0):
    t = int(sum(new)) + extra
    tab = torch.full((len(ctx), table.shape[1] + wide), -5, dtype=torch.int32)
    tab[:, wide // 2: wide // 2 + table.shape[1]] = torch.from_numpy(table)
    tab = tab.cuda()
    view = tab[:, wide // 2: wide // 2 + table.shape[1]]
    c, left = i32(ctx).cuda(), i32([n_free]).cuda()
    kw = dict(seq_lens=c, n_free_out=left) if in_place else {}
    lens, slots, left = G.gdn_cache_plan(c, page, view, torch.from_numpy(free).cuda(), left, cu_seqlens=None if cu is None else cu_of(new, cu).cuda(),
                                         n_tokens=t, **kw)
    torch.cuda.synchronize()
    assert wide == 0 or ((tab[:, : wide // 2] == -5).all() and (tab[:, wide // 2 + table.shape[1]:] == -5).all())
    starts = np.concatenate([[0], np.cumsum(new)]).astype(int)
    want = A.plan(list(ctx), starts, table, free, max(0, min(n_free, len(free))), page, t)
    for name, got, ref in zip(("table", "lens", "slots"), (view, lens, slots), want):
        assert np.array_equal(got.cpu().numpy(), ref), name
    assert int(left) == want[3]
    return want


@pytest.mark.parametrize("page", [1, 16, 48, 1000])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("seqs,most,supply", [(1, 5, 1.0), (3, 40, 0.5), (64, 300, 1.0), (64, 300, 0.6), (700, 20, 0.9), (1500, 4, 0.5)])
def test_plan(page, in_place, seqs, most, supply):
    rng = np.random.default_rng(seqs + page)
    ctx, new = rng.integers(0, most, seqs), rng.integers(0, most, seqs)
    width = int(-(-(2 * most) // page))
    table, free = tables(rng, ctx, width, page, seqs * width)
    wanted = sum(-(-(a + b) // page) - -(-a // page) for a, b in zip(ctx, new))
    run_plan(ctx, new, table, free, int(wanted * supply), page, extra=5, in_place=in_place, wide=6)


@pytest.mark.parametrize("cu", [None, torch.int32, torch.int64])
@pytest.mark.parametrize("seqs", [1, 256, 3000])
def test_plan_one_token_each(seqs, cu):
    rng = np.random.default_rng(seqs)
    ctx = rng.integers(0, 100, seqs)
    table, free = tables(rng, ctx, 7, 16, seqs)
    run_plan(ctx, [1] * seqs, table, free, seqs, 16, cu=cu)


def test_plan_tables_without_room():
    rng = np.random.default_rng(5)
    ctx, new = [30, 10, 31, 0, 40], [3, 2, 1, 33, 0]
    table, free = tables(rng, ctx, 4, 8, 20)   # 32 tokens a row
    want = run_plan(ctx, new, table, free, 20, 8)
    assert want[1].tolist() == [30, 12, 32, 0, 40]


@pytest.mark.parametrize("n_free", [-3, 0, 10 ** 6])
def test_plan_counts_outside_the_stack(n_free):
    rng = np.random.default_rng(6)
    ctx, new = [3, 16, 9], [4, 4, 40]
    table, free = tables(rng, ctx, 5, 16, 6)
    run_plan(ctx, new, table, free, n_free, 16)


def test_plan_malformed_starts_and_lengths_stay_in_range():
    table, free = torch.zeros(3, 4, dtype=torch.int32).cuda(), torch.arange(8, dtype=torch.int32).cuda()
    for cu in ([0, 50, 20, 70], [9, 9, 10 ** 9, -1], [-9, 0, 0, 60]):
        for ctx in ([0, 0, 0], [-7, 2 ** 31 - 1, 3]):
            lens, slots, left = G.gdn_cache_plan(i32(ctx).cuda(), 16, table, free, i32([8]).cuda(), cu_seqlens=i32(cu).cuda(), n_tokens=60)
            assert 0 <= int(left) <= 8 and int(slots.max()) < 8 * 16 and int(slots.min()) >= -1


def test_plan_without_requests_or_tokens():
    lens, slots, left = G.gdn_cache_plan(i32([5, 0]).cuda(), 16, torch.zeros(2, 3, dtype=torch.int32).cuda(), i32([4]).cuda(), i32([1]).cuda(),
                                         cu_seqlens=i32([0, 0, 0]).cuda(), n_tokens=0)
    assert lens.tolist() == [5, 0] and slots.numel() == 0 and int(left) == 1


@pytest.mark.parametrize("seqs", [1, 5, 600, 1100])
@pytest.mark.parametrize("room", [0, 10 ** 6])
def test_release(seqs, room):
    rng = np.random.default_rng(seqs)
    page, width = 16, 9
    lens = rng.integers(0, page * width + 1, seqs)
    done = rng.integers(0, 2, seqs)
    table, free = tables(rng, lens, width, page, 7)
    stack = np.full(len(free) + min(room, int(table.max()) + 1), -1, np.int32)
    stack[: len(free)] = free
    if room == 0:
        stack = stack[:]
    want = A.release(done, lens.astype(np.int32), table, stack, 5, page)
    t, l, f, n = torch.from_numpy(table).cuda(), i32(lens).cuda(), torch.from_numpy(stack).cuda(), i32([5]).cuda()
    G.gdn_cache_release(i32(done).cuda(), l, page, t, f, n)
    for name, got, ref in zip(("lens", "table", "free"), (l, t, f), want):
        assert np.array_equal(got.cpu().numpy(), ref), name
    assert int(n) == want[3]


@pytest.mark.parametrize("dtype", dtypes)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Hk,page,T", [(1, 16, 1), (8, 16, 37), (3, 7, 500), (2, 1, 64)])
@pytest.mark.parametrize("form", ["plain", "head-major", "interleaved"])
def test_store(dtype, d, Hk, page, T, form):
    g, dt = gen(d + T), dtypes[dtype]
    pages = -(-T // page) + 4
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[::5] = torch.tensor([-1, pages * page, 2 ** 40, -2 ** 62])[torch.arange(slots[::5].numel()) % 4]
    rows = randn(g, T, 3 * Hk * d, dtype=dt)
    base = randn(g, 2, pages, page, Hk, d, dtype=dt)
    rg = rows.cuda()
    k, v = (rg[:, i * Hk * d: (i + 1) * Hk * d].view(T, Hk, d) for i in (0, 2))
    if form == "plain":
        kc, vc = base[0].cuda(), base[1].cuda()
    elif form == "head-major":
        kc, vc = (x.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3) for x in base)
    else:
        both = base.permute(1, 0, 2, 3, 4).contiguous().cuda()
        kc, vc = both[:, 0], both[:, 1]
    G.gdn_cache_store(k, v, slots.cuda(), kc, vc)
    ok = (slots >= 0) & (slots < pages * page)
    for got, want, src in ((kc, base[0], rows[:, : Hk * d]), (vc, base[1], rows[:, 2 * Hk * d:])):
        want = want.clone().view(pages * page, Hk, d)
        want[slots[ok]] = src.reshape(T, Hk, d)[ok]
        assert torch.equal(got.cpu().reshape(pages * page, Hk, d), want)


def test_a_life_of_requests():
    """Prompts, steps, releases: pages are never in two places at once, and
    the stack gets all of them back."""
    rng = np.random.default_rng(9)
    N, page, width, pages = 12, 8, 20, 90
    table, lens = torch.full((N, width), -1, dtype=torch.int32).cuda(), torch.zeros(N, dtype=torch.int32).cuda()
    free, n = torch.randperm(pages, generator=gen(1)).to(torch.int32).cuda(), i32([pages]).cuda()
    for turn in range(30):
        new = rng.integers(0, 12, N) * rng.integers(0, 2, N)
        t = int(new.sum())
        G.gdn_cache_plan(lens, page, table, free, n, cu_seqlens=cu_of(new).cuda(), n_tokens=t, seq_lens=lens, n_free_out=n)
        done = rng.integers(0, 6, N) == 0
        G.gdn_cache_release(i32(done).cuda(), lens, page, table, free, n)
        l, tab = lens.cpu().numpy(), table.cpu().numpy()
        held = [tab[i, j] for i in range(N) for j in range(-(-int(l[i]) // page))]
        every = sorted(held + free.cpu().tolist()[: int(n)])
        assert every == list(range(pages)), turn
    G.gdn_cache_release(i32([1] * N).cuda(), lens, page, table, free, n)
    assert int(n) == pages and int(lens.abs().sum()) == 0
