"""The attention over a paged cache as a program runs it: a service's life of
requests against the whole sequences' attention, steps captured into graphs,
streams and threads side by side, caches past 4 GiB, and caches of nothing."""
import threading

import numpy as np
import pytest
import torch

import gated_deltanet_02_amd as G
from tests.attn_util import A, check_out, cu_of, dtypes, f64, gen, make_pool, randn, reference

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32)


@pytest.mark.parametrize("dtype,d,page,window,sinks", [(torch.bfloat16, 128, 16, 0, 0), (torch.bfloat16, 64, 48, 70, 3), (torch.bfloat16, 256, 64, 0, 0),
                                                       (torch.float32, 64, 16, 33, 0)])
def test_a_service_of_requests(dtype, d, page, window, sinks):
    """Requests come, are read in chunks beside others' single tokens, grow
    and leave, their pages used again: every row against the attention over
    the tokens that its request has seen."""
    N, H, Hk, width, pages = 5, 6, 2, 40, 200
    rng, g = np.random.default_rng(d + page), gen(d)
    kc, vc = (torch.full((pages, page, Hk, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    table, lens = torch.full((N, width), -1, dtype=torch.int32, device="cuda"), torch.zeros(N, dtype=torch.int32, device="cuda")
    free, left = torch.randperm(pages, generator=g).to(torch.int32).cuda(), i32([pages]).cuda()
    past = [[torch.empty(0, Hk, d, dtype=dtype) for _ in range(2)] for _ in range(N)]
    for turn in range(10):
        if turn % 2 == 0:  # chunks of prompts, some of nothing
            new = [int(n) for n in rng.integers(0, 200, N) * rng.integers(0, 2, N)]
        else:  # a step of all
            new = [1] * N
        t = sum(new)
        q, k, v = randn(g, t, H, d, dtype=dtype), randn(g, t, Hk, d, dtype=dtype), randn(g, t, Hk, d, dtype=dtype)
        before = left.item()
        _, slots, _ = G.gdn_cache_plan(lens, page, table, free, left, cu_seqlens=cu_of(new).cuda() if turn % 2 == 0 else None, n_tokens=t, seq_lens=lens,
                                       n_free_out=left)
        assert before - left.item() == sum(-(-(len(past[i][0]) + new[i]) // page) - -(-len(past[i][0]) // page) for i in range(N))
        G.gdn_cache_store(k.cuda(), v.cuda(), slots, kc, vc)
        if turn % 2 == 0:
            out = G.gdn_attn_prefill(q.cuda(), kc, vc, cu_seqlens=cu_of(new).cuda(), block_table=table, seq_lens=lens, window=window, sinks=sinks)
        else:
            out = G.gdn_attn_decode(q.cuda(), kc, vc, table, lens, window=window, sinks=sinks)
        starts = np.concatenate([[0], np.cumsum(new)])
        for i in range(N):
            a, b = int(starts[i]), int(starts[i + 1])
            past[i] = [torch.cat([old, x[a:b]]) for old, x in zip(past[i], (k, v))]
            if b > a:
                ref = A.attention(f64(q[a:b]), f64(past[i][0]), f64(past[i][1]), len(past[i][0]) - (b - a), window, sinks, None)
                check_out(out[a:b], ref, dtype, f"turn {turn} request {i}", step=turn % 2 == 1)
        assert lens.tolist() == [len(p[0]) for p in past]
        done = (rng.integers(0, 4, N) == 0) | (np.array([len(p[0]) for p in past]) > 400)
        G.gdn_cache_release(i32(done).cuda(), lens, page, table, free, left)
        for i in np.nonzero(done)[0]:
            past[i] = [x[:0] for x in past[i]]


def steps(n, lens, H, Hk, d, dtype, page, seed):
    """n steps of running sequences: a function that runs them from the state
    that `reset` sets, and their outputs."""
    g = gen(seed)
    N = len(lens)
    k0, v0, tab0, spare = make_pool(g, lens, page, Hk, d, dtype, spare=N * (n // page + 2), width=max(lens) // page + n // page + 3)
    rows = [[randn(g, N, heads, d, dtype=dtype).cuda() for heads in (H, Hk, Hk)] for _ in range(n)]
    state = dict(k=k0.cuda(), v=v0.cuda(), table=tab0.cuda(), lens=i32(lens).cuda(), free=spare.cuda(), left=i32([len(spare)]).cuda())
    first = {x: y.clone() for x, y in state.items()}
    outs = [torch.empty_like(r[0]) for r in rows]
    slots = torch.empty(N, dtype=torch.int64, device="cuda")

    def reset():
        for x, y in first.items():
            state[x].copy_(y)
        for o in outs:
            o.fill_(9.0)

    def run(ws):
        s = state
        for (q, k, v), o in zip(rows, outs):
            G.gdn_cache_plan(s["lens"], page, s["table"], s["free"], s["left"], seq_lens=s["lens"], slots=slots, n_free_out=s["left"])
            G.gdn_cache_store(k, v, slots, s["k"], s["v"])
            G.gdn_attn_decode(q, s["k"], s["v"], s["table"], s["lens"], out=o, workspace=ws)

    return reset, run, outs, state


def capture(run, ws):
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph):
            run(ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    return graph


def test_steps_in_two_graphs_that_share_a_workspace():
    cases = [steps(5, [1, 300, 64, 2000], 8, 2, 128, torch.bfloat16, 16, 1), steps(4, [7000], 4, 1, 128, torch.bfloat16, 64, 2)]
    ws = torch.empty(G.gdn_attn_workspace_size(cases[0][2][0]), dtype=torch.uint8, device="cuda")
    want, graphs = [], []
    for reset, run, outs, state in cases:
        reset()
        run(ws)
        torch.cuda.synchronize()
        want.append([o.clone() for o in outs] + [state[x].clone() for x in ("table", "lens", "left", "k", "v")])
        reset()
        graphs.append(capture(run, ws))
    for rep in range(3):
        for reset, *_ in cases:
            reset()
        ws.fill_(255)
        torch.cuda.synchronize()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for (_, _, outs, state), ref in zip(cases, want):
            for a, b in zip(outs + [state[x] for x in ("table", "lens", "left", "k", "v")], ref):
                assert torch.equal(a, b), f"replay {rep}"
        cases[0][0]()
        cases[0][1](ws)  # eager work of the program between replays


def test_a_prompt_in_a_captured_graph():
    g = gen(3)
    lengths = [700, 0, 33, 1500]
    t, cu = sum(lengths), cu_of(lengths).cuda()
    q, k, v = randn(g, t, 8, 128, dtype=torch.bfloat16).cuda(), randn(g, t, 2, 128, dtype=torch.bfloat16).cuda(), randn(g, t, 2, 128, dtype=torch.bfloat16).cuda()
    want, out = G.gdn_attn_prefill(q, k, v, cu_seqlens=cu), torch.empty_like(q)
    graph = capture(lambda _: G.gdn_attn_prefill(q, k, v, cu_seqlens=cu, out=out), None)
    for rep in range(3):
        out.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), rep
        assert torch.equal(G.gdn_attn_prefill(q, k, v, cu_seqlens=cu), want)


def test_streams_and_threads_side_by_side():
    """Two threads, each on a stream of its own, with inputs, outputs and a
    workspace of its own: the results of one after the other, bit for bit."""
    cases = [steps(6, [1, 500, 64, 2000], 8, 2, 64, torch.bfloat16, 16, 4), steps(6, [900, 3], 4, 2, 256, torch.float32, 48, 5)]
    spaces = [torch.empty(G.gdn_attn_workspace_size(c[2][0]), dtype=torch.uint8, device="cuda") for c in cases]
    want = []
    for (reset, run, outs, _), ws in zip(cases, spaces):
        reset()
        run(ws)
        torch.cuda.synchronize()
        want.append([o.clone() for o in outs])
        reset()
    torch.cuda.synchronize()
    errors = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(5):
                    cases[i][0]()
                    cases[i][1](spaces[i])
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not errors
    for (_, _, outs, _), ref in zip(cases, want):
        for a, b in zip(outs, ref):
            assert torch.equal(a, b)


def test_a_stream_that_is_named():
    g = gen(6)
    k, v, table, _ = make_pool(g, [100, 40], 16, 2, 64, torch.bfloat16)
    q = randn(g, 2, 4, 64, dtype=torch.bfloat16).cuda()
    args = (k.cuda(), v.cuda(), table.cuda(), i32([100, 40]).cuda())
    want = G.gdn_attn_decode(q, *args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = G.gdn_attn_decode(q, *args, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype,d,page", [(torch.bfloat16, 128, 16), (torch.bfloat16, 64, 48), (torch.float32, 128, 16)])
def test_caches_past_four_gib(dtype, d, page):
    """Pages on both sides of 2^31 elements and of 2^32 bytes."""
    Hk, H, lens = 2, 4, [500, 130]
    row = Hk * d
    pages = (1 << 31) // (page * row) + 40  # (a little over 2^31 elements)
    kc, vc = (torch.empty(pages, page, Hk, d, dtype=dtype, device="cuda") for _ in range(2))
    have = [-(-n // page) for n in lens]
    at4 = (1 << 32) // (page * row * kc.element_size())
    near = sorted({p + o for p in (pages - 40, at4) for o in range(-6, 7)} | {0, pages - 1} | set(range(100, 140)))
    order = torch.tensor(near)[torch.randperm(len(near), generator=gen(7))][: sum(have)]
    assert len(set(order.tolist())) == sum(have) and int(order.max()) >= pages - 40
    table = torch.full((2, max(have)), -1, dtype=torch.int32)
    table[0, : have[0]], table[1, : have[1]] = order[: have[0]].int(), order[have[0]:].int()
    g = gen(8)
    k, v = randn(g, sum(lens), Hk, d, dtype=dtype), randn(g, sum(lens), Hk, d, dtype=dtype)
    slots = torch.cat([table[i, torch.arange(n) // page].long() * page + torch.arange(n) % page for i, n in enumerate(lens)])
    G.gdn_cache_store(k.cuda(), v.cuda(), slots.cuda(), kc, vc)
    for got, want in ((kc, k), (vc, v)):
        flat = got.view(pages * page, Hk, d)
        assert torch.equal(torch.stack([flat[int(s)] for s in slots[::37]]).cpu(), want[::37])
    q = randn(g, sum(lens), H, d, dtype=dtype)
    out = G.gdn_attn_prefill(q.cuda(), kc, vc, cu_seqlens=cu_of(lens).cuda(), block_table=table.cuda(), seq_lens=i32(lens).cuda())
    last = torch.tensor([lens[0] - 1, sum(lens) - 1])
    one = G.gdn_attn_decode(q[last].cuda(), kc, vc, table.cuda(), i32(lens).cuda())
    for i, (a, b) in enumerate(((0, lens[0]), (lens[0], sum(lens)))):
        ref = A.attention(f64(q[a:b]), f64(k[a:b]), f64(v[a:b]), 0, 0, 0, None)
        check_out(out[a:b], ref, dtype, f"prompt {i}")
        check_out(one[i: i + 1], tuple(x[-1:] for x in ref), dtype, f"step {i}", step=True)


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.bfloat16, 256), (torch.float32, 64)])
def test_tokens_far_apart(dtype, d):
    """Rows of prompts whose offsets pass 2^31 elements."""
    T, Hk, far = 700, 2, 1 << 22
    wide = torch.empty(T * far, dtype=dtype, device="cuda")
    g = gen(9)
    k, v, q = randn(g, T, Hk, d, dtype=dtype), randn(g, T, Hk, d, dtype=dtype), randn(g, T, 4, d, dtype=dtype)
    kw, vw = wide.as_strided((T, Hk, d), (far, d, 1)), wide.as_strided((T, Hk, d), (far, d, 1), 4096)
    kw.copy_(k.cuda())
    vw.copy_(v.cuda())
    out = wide.as_strided((T, 4, d), (far, d, 1), 16384)
    got = G.gdn_attn_prefill(q.cuda(), kw, vw)
    check_out(got, A.attention(f64(q), f64(k), f64(v), 0, 0, 0, None), dtype, "out")
    with pytest.raises(G.GdnError):
        G.gdn_attn_prefill(q.cuda(), kw, vw, out=out)  # (its range covers the keys')


@pytest.mark.parametrize("dtype", list(dtypes.values()), ids=list(dtypes))
def test_caches_of_nothing(dtype):
    """No pages, or tables of no width: no query sees anything."""
    q, lens, cu = randn(gen(10), 5, 4, 64, dtype=dtype).cuda(), i32([0, 9]).cuda(), cu_of([2, 3]).cuda()
    for pages, width in ((0, 4), (3, 0), (0, 0)):
        c = torch.full((pages, 16, 2, 64), float("nan"), dtype=dtype, device="cuda")
        table = torch.zeros(2, width, dtype=torch.int32, device="cuda")
        out = G.gdn_attn_prefill(q, c, c, cu_seqlens=cu, block_table=table, seq_lens=lens)
        one = G.gdn_attn_decode(q[:2], c, c, table, lens)
        torch.cuda.synchronize()
        assert not out.any() and not one.any()


@pytest.mark.parametrize("dtype", list(dtypes.values()), ids=list(dtypes))
def test_uniform_batch_behind_a_cache(dtype):
    g, lens = gen(11), [200, 64, 131]
    k, v, table, _ = make_pool(g, lens, 16, 2, 128, dtype, fill=float("nan"))
    q = randn(g, 3, 40, 4, 128, dtype=dtype)
    out = G.gdn_attn_prefill(q.cuda(), k.cuda(), v.cuda(), block_table=table.cuda(), seq_lens=i32(lens).cuda())
    ref = reference(q.reshape(120, 4, 128), k, v, table, lens, [0, 40, 80, 120])
    check_out(out.reshape(120, 4, 128), ref, dtype, "out")


@pytest.mark.parametrize("dtype", list(dtypes.values()), ids=list(dtypes))
@pytest.mark.parametrize("d", [64, 128, 256])
def test_nothing_passes_between_sequences_or_from_behind_them(dtype, d):
    """NaN and infinities in a sequence's keys and values, in its neighbours'
    queries and behind the batch stay where they are."""
    g, lengths = gen(12), [70, 130, 1, 60]
    t = sum(lengths)
    q, k, v = randn(g, t + 9, 4, d, dtype=dtype), randn(g, t + 9, 2, d, dtype=dtype), randn(g, t + 9, 2, d, dtype=dtype)
    for x in (q, k, v):
        x[70:200] = float("nan")
        x[t:] = float("inf")
    out = torch.full((t + 9, 4, d), 5.0, dtype=dtype, device="cuda")
    G.gdn_attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu_seqlens=cu_of(lengths).cuda(), out=out)
    assert (out[t:] == 5.0).all() and out[70:200].isnan().all()
    for a, b in ((0, 70), (200, 201), (201, t)):
        check_out(out[a:b], A.attention(f64(q[a:b]), f64(k[a:b]), f64(v[a:b]), 0, 0, 0, None), dtype, f"rows {a}")


def test_keys_of_minus_infinity():
    """Scores of -inf weigh nothing beside others, and rows of nothing else are
    not a number, as the formula has it, or zero; never anything else."""
    for d in (64, 128, 256):
        q, k, v = torch.ones(200, 2, d), torch.ones(200, 2, d) * 0.01, randn(gen(13), 200, 2, d)
        k[10:150, 0, 0] = -float("inf")
        q, k, v = (x.bfloat16() for x in (q, k, v))
        out = G.gdn_attn_prefill(q.cuda(), k.cuda(), v.cuda())
        torch.cuda.synchronize()
        seen = [j for j in range(200) if not 10 <= j < 150]
        for h, keys in ((0, seen), (1, list(range(200)))):
            ref = A.attention(f64(q[199:, h: h + 1]), f64(k[keys][:, h: h + 1]), f64(v[keys][:, h: h + 1]), len(keys) - 1, 0, 0, None)
            check_out(out[199:, h: h + 1], ref, torch.bfloat16, f"head {h} d {d}")


def test_as_many_requests_as_there_may_be():
    """2^20 requests: a token planned for each, and 70000 sequences of which
    most are short or empty, single tokens on them."""
    n, page = 1 << 20, 16
    rng = np.random.default_rng(14)
    ctx = rng.integers(0, 40, n)
    have, need = -(-ctx // page), -(-(ctx + 1) // page)
    extra = need - have
    upto = np.cumsum(extra)
    supply = int(upto[-1]) - 1000  # (the last ones get none)
    held = np.arange(n * 3, dtype=np.int32).reshape(n, 3)
    table = np.where(np.arange(3) < have[:, None], held, -1)
    free = np.arange(supply, dtype=np.int32) + 5 * n
    tab = torch.from_numpy(table).cuda()
    lens, slots, left = G.gdn_cache_plan(i32(ctx).cuda(), page, tab, torch.from_numpy(free).cuda(), i32([supply]).cuda())
    served = (extra == 0) | (upto <= supply)
    pick = np.clip(supply - upto, 0, supply - 1)  # (a page each)
    want_page = np.where(extra > 0, free[pick], table[np.arange(n), ctx // page])
    want = np.where(served, want_page.astype(np.int64) * page + ctx % page, -1)
    assert np.array_equal(slots.cpu().numpy(), want)
    assert np.array_equal(lens.cpu().numpy(), np.where(served, ctx + 1, ctx))
    assert int(left) == supply - int(upto[served & (extra > 0)].max())

    N, d = 70000, 64
    g = gen(15)
    lens = torch.randint(0, 4, (N,), generator=g).int()
    lens[torch.rand(N, generator=g) < 0.3] = 0
    lens[40000], lens[N - 1] = 900, 70
    width, pg = 4, 256
    k, v = randn(g, N // 8, pg, 1, d), randn(g, N // 8, pg, 1, d)
    table = torch.randint(0, N // 8, (N, width), generator=g).int()
    q = randn(g, N, 2, d)
    out = G.gdn_attn_decode(q.cuda(), k.cuda(), v.cuda(), table.cuda(), lens.cuda()).cpu()
    assert not out[lens == 0].any()
    some = torch.cat([torch.tensor([40000, N - 1]), torch.nonzero(lens > 0)[::301, 0]]).tolist()
    kd, vd = f64(k), f64(v)
    for i in some:
        m = int(lens[i])
        ref = A.attention(f64(q[i: i + 1]), A.gather(kd, table[i].tolist(), m), A.gather(vd, table[i].tolist(), m), m - 1, 0, 0, None)
        check_out(out[i: i + 1], ref, torch.float32, f"sequence {i}", step=True)
