"""The attention's kernels in every form that a call can choose: few (tile,
head) pairs, whose keys are shared between groups of waves, and many; rows and
pages, of sizes that keep a copy's rows together and that do not; windows and
none; every d and type."""
import pytest

from tests.attn_util import dtypes
from tests.test_gpu_attn import decode, prefill, pytestmark  # noqa: F401

LENGTHS, PAST = [200, 0, 330, 9, 65], [0, 40, 300, 65, 511]
# (604 tokens, 5 sequences: 36 and 576 pairs of 128 queries and a head, 56 and 896 of 64)
HEADS = [4, 64]
WINDOWS = [(0, 0), (1, 0), (33, 4), (100, 70), (300, 1), (5000, 2)]


@pytest.mark.parametrize("dtype", dtypes)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H", HEADS)
@pytest.mark.parametrize("page", [12, 16])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_prefill_behind_a_cache(dtype, d, H, page, window, sinks):
    prefill(page + H, LENGTHS, H, 2, d, dtypes[dtype], window=window, sinks=sinks, past=PAST, page=page, extra=2)


@pytest.mark.parametrize("dtype", dtypes)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H", HEADS)
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_prefill_of_rows(dtype, d, H, window, sinks):
    prefill(H, LENGTHS, H, 2, d, dtypes[dtype], window=window, sinks=sinks, extra=2)


@pytest.mark.parametrize("dtype", dtypes)
@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("page", [12, 16])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (33, 4), (100, 64), (100, 1), (5000, 3), (64, 5000)])
def test_decode_windows(dtype, d, page, window, sinks):
    lens = [0, 1, 2, 5, 15, 16, 17, 40, 99, 100, 101, 104, 164, 165, 1300]
    decode(window + sinks, lens, 20, 1, d, dtypes[dtype], page, window=window, sinks=sinks)
