"""Release of requests whose rows of the table name pages and, in places,
none: what goes back onto the stack is pages alone, so that the next plan hands
out nothing else."""
import numpy as np
import pytest
import torch

import gated_deltanet_02_amd as G
from tests.attn_util import A, cu_of

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32)


def test_a_released_row_without_a_page_gives_no_page():
    """A row of [none, 1], released; the 32 tokens of the next request need two
    pages of 16 where one is on the stack: the request waits."""
    table, lens = i32([[-1, 1], [7, 7]]).cuda(), i32([32, 0]).cuda()
    free, left = i32([9, 9, 9]).cuda(), i32([0]).cuda()
    G.gdn_cache_release(i32([1, 0]).cuda(), lens, 16, table, free, left)
    assert int(left) == 1 and free.tolist() == [1, 9, 9] and table[0].tolist() == [-1, -1]
    lens, slots, left = G.gdn_cache_plan(lens, 16, table, free, left, cu_seqlens=cu_of([0, 32]).cuda(), n_tokens=32)
    assert lens.tolist() == [0, 0] and (slots == -1).all() and int(left) == 1


@pytest.mark.parametrize("seqs,width", [(1, 1), (5, 9), (64, 63), (65, 64), (600, 65), (520, 130), (1100, 9), (5, 1300), (40, 600), (1, 5000)])
@pytest.mark.parametrize("none", [0.0, 0.3, 1.0])
@pytest.mark.parametrize("room", [0, 37, 10 ** 6])
def test_release_passes_over_entries_without_a_page(seqs, width, none, room):
    rng = np.random.default_rng(seqs + width)
    page, wide = 16, width + 5
    lens = rng.integers(-3, page * width + 40, seqs)  # (some past the table's end)
    done = rng.integers(0, 3, seqs) - 1               # any number but 0 is done
    table = rng.permutation(seqs * width).reshape(seqs, width).astype(np.int32)
    table[rng.random(table.shape) < none] = -1
    table[(table >= 0) & (rng.random(table.shape) < none / 4)] = -2 ** 31
    stack = np.full(11 + min(room, table.size), -9, np.int32)
    stack[:11] = seqs * width + np.arange(11)
    want = A.release(done, np.maximum(lens, 0).astype(np.int32), table, stack, 11, page)
    want[0][done == 0] = lens[done == 0]
    t = torch.full((seqs, wide), -7, dtype=torch.int32)
    t[:, 2: 2 + width] = torch.from_numpy(table)
    t = t.cuda()
    l, f, n = i32(lens).cuda(), torch.from_numpy(stack).cuda(), i32([11]).cuda()
    G.gdn_cache_release(i32(done).cuda(), l, page, t[:, 2: 2 + width], f, n)
    for name, got, ref in zip(("lens", "table", "free"), (l, t[:, 2: 2 + width], f), want):
        assert np.array_equal(got.cpu().numpy(), ref), name
    assert int(n) == want[3]
    assert (t[:, :2] == -7).all() and (t[:, 2 + width:] == -7).all()


def test_pages_given_up_behind_a_window_are_not_released_again():
    """A request whose first pages its owner has put back already."""
    table, lens = torch.arange(8, dtype=torch.int32).view(1, 8).cuda(), i32([120]).cuda()
    free, left = torch.full((8,), -1, dtype=torch.int32).cuda(), i32([3]).cuda()
    free[:3] = table[0, :3]
    table[0, :3] = -1
    G.gdn_cache_release(i32([1]).cuda(), lens, 16, table, free, left)
    assert int(left) == 8 and sorted(free.tolist()) == list(range(8))
