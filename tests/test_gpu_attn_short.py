"""A stack of free pages that is too short, run through to the attention: rows
with a slot are right, those of requests that wait are known by their slots,
and nothing of theirs is stored, until a later plan serves them."""
import numpy as np
import pytest
import torch

import gated_deltanet_02_amd as G
from tests.attn_util import A, check_out, cu_of, f64, gen, randn

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32)


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float32, 64), (torch.bfloat16, 256)])
@pytest.mark.parametrize("single", [False, True])
def test_requests_wait_for_pages(dtype, d, single):
    N, H, Hk, page, width, pages = 6, 4, 2, 16, 12, 19 if single else 22
    rng, g = np.random.default_rng(d + single), gen(d)
    kc, vc = (torch.full((pages, page, Hk, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    table, lens = torch.full((N, width), -1, dtype=torch.int32, device="cuda"), torch.zeros(N, dtype=torch.int32, device="cuda")
    free, left = torch.randperm(pages, generator=g).to(torch.int32).cuda(), i32([pages]).cuda()
    past = [[torch.empty(0, Hk, d, dtype=dtype) for _ in range(2)] for _ in range(N)]
    waited, came_back, waits = 0, 0, [False] * N
    for turn in range(14):
        prompt = not single or turn == 0
        new = [int(n) for n in rng.integers(1, 70, N)] if prompt else [1] * N
        if single and turn == 0:  # all pages' last places: every step needs pages
            new = [page * (2 + (i < 4)) for i in range(N)]
        t, starts = sum(new), np.concatenate([[0], np.cumsum(new)])
        q, k, v = randn(g, t, H, d, dtype=dtype), randn(g, t, Hk, d, dtype=dtype), randn(g, t, Hk, d, dtype=dtype)
        cu = cu_of(new).cuda() if prompt else None
        _, slots, _ = G.gdn_cache_plan(lens, page, table, free, left, cu_seqlens=cu, n_tokens=t, seq_lens=lens, n_free_out=left)
        G.gdn_cache_store(k.cuda(), v.cuda(), slots, kc, vc)
        if prompt:
            out = G.gdn_attn_prefill(q.cuda(), kc, vc, cu_seqlens=cu, block_table=table, seq_lens=lens)
        else:
            out = G.gdn_attn_decode(q.cuda(), kc, vc, table, lens)
        served = (slots >= 0).cpu()
        kept = torch.where(served.cuda()[:, None, None], out, 0)
        for i in range(N):
            a, b = int(starts[i]), int(starts[i + 1])
            assert served[a:b].all() or not served[a:b].any(), "all of a request's tokens or none"
            if not served[a]:
                waited, waits[i] = waited + 1, True
                assert int(lens[i]) == len(past[i][0]) and (kept[a:b] == 0).all()
                continue
            came_back, waits[i] = came_back + waits[i], False
            past[i] = [torch.cat([old, x[a:b]]) for old, x in zip(past[i], (k, v))]
            ref = A.attention(f64(q[a:b]), f64(past[i][0]), f64(past[i][1]), len(past[i][0]) - (b - a))
            check_out(kept[a:b], ref, dtype, f"turn {turn} request {i}", step=not prompt)
        assert lens.tolist() == [len(p[0]) for p in past]
        if turn % 3 == 2:  # the longest one leaves
            out_of = int(np.argmax([len(p[0]) for p in past]))
            G.gdn_cache_release(i32([i == out_of for i in range(N)]).cuda(), lens, page, table, free, left)
            past[out_of] = [x[:0] for x in past[out_of]]
    assert waited > 0 and came_back > 0
