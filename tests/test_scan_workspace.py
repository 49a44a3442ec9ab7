"""What the scan's workspace holds (host only): states only for sequences that
can be cut, whatever the number of others beside them."""
import ctypes
import os

import pytest

from gated_deltanet_02_amd import _binding as B
from gated_deltanet_02_amd import _layer as L
from tests.test_layer_boundary import BF16, F32, I32, expect, fake, opts, ref


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.library_path()):
        pytest.fail("libgdn.so is not built (run __graft_entry__.build())")
    return L._functions()


def size(lib, T, H, G, N, P, n_seq=None, segment_blocks=0, dtype=BF16):
    n = ctypes.c_size_t(0)
    x, b = fake((T, H, P), dtype), fake((T, G, N), dtype)
    cu = None if n_seq is None else fake((n_seq + 1,), I32)
    expect(lib.gdn_ssm_workspace_size(ref(x), ref(b), ref(cu), ref(opts(segment_blocks=segment_blocks)), ctypes.byref(n)), 0)
    return n.value


def up(v):
    return (v + 255) // 256 * 256


@pytest.mark.parametrize("H,N,P", [(16, 128, 128), (48, 16, 64)])
@pytest.mark.parametrize("n,each", [(256, 128), (4096, 16), (3, 4096), (1, 65), (64, 65), (1000, 64), (1 << 20, 1)])
@pytest.mark.parametrize("blocks", [1, 2, 64])
def test_packed_batches(lib, H, N, P, n, each, blocks):
    """Of n sequences of T tokens in all, at most T / (s + 1) have more than s
    tokens, with at most T / s and one segment each; a slot for each segment
    and one for each such sequence."""
    T, s = n * each, 64 * blocks
    want = up(16 * (T // s + n)) + up(4 * (n + 1))
    if T > s:
        cuts = min(n, T // (s + 1))
        segs = T // s + cuts
        slots = segs + cuts
        want += up(16 * (cuts + 1)) + up(16 * segs) + up(4 * slots * H) + up(4 * slots * H * N * P)
    if (T // s + n + 7) * H * 4 * P < 1 << 32 and n * H < 1 << 24:
        assert size(lib, T, H, 1, N, P, n, blocks) == want


@pytest.mark.parametrize("T,H,n", [(256 * 128, 16, 256), (4096 * 16, 48, 4096), (1 << 20, 16, 1 << 14)])
def test_many_short_prompts_need_little(lib, T, H, n):
    """Less than a quarter of the states that the batch carries itself."""
    assert size(lib, T, H, 1, 128, 128, n) < n * H * 128 * 128 * 4 / 4


@pytest.mark.parametrize("B,T", [(1, 640), (3, 640), (7, 65)])
def test_uniform_batches(lib, B, T):
    n = ctypes.c_size_t(0)
    x, b = fake((B, T, 4, 32), F32), fake((B, T, 2, 64), F32)
    expect(lib.gdn_ssm_workspace_size(ref(x), ref(b), None, ref(opts(segment_blocks=1)), ctypes.byref(n)), 0)
    slots = B * (-(-T // 64) + 1)
    assert n.value == up(4 * slots * 4) + slots * 4 * 64 * 32 * 4


@pytest.mark.parametrize("T", [1 << 20, (1 << 20) + 1, 1 << 24, (1 << 31) - (1 << 21)])
@pytest.mark.parametrize("blocks", [-1, 1 << 25, (1 << 31) - 1])
def test_one_pass_over_long_sequences(lib, T, blocks):
    """Nothing is cut, however long: no states, of packed ones the table."""
    assert size(lib, T, 1, 1, 16, 16, None, blocks) == 0
    assert size(lib, T, 1, 1, 16, 16, 3, blocks) == up(16 * 4) + up(4 * 4)
    # and segments of that many blocks where there are more
    assert size(lib, T, 1, 1, 16, 16, None, 1 << 14) == (0 if T == 1 << 20 else up(4 * (-(-T // (1 << 20)) + 1)) + (-(-T // (1 << 20)) + 1) * 1024)
