"""Arguments of the attention's binding that are refused before any tensor is
looked at (no GPU needed)."""
import numpy as np
import pytest
import torch

import gated_deltanet_02_amd as G
from oracle import attention as A


def test_a_scale_of_zero_is_refused():
    """0 is how the C ABI names the default: it must not pass for one."""
    x, c, t = torch.randn(4, 2, 64), torch.randn(3, 16, 2, 64), torch.zeros(4, 2, dtype=torch.int32)
    for zero in (0, 0.0, -0.0):
        with pytest.raises(ValueError, match="scale"):
            G.gdn_attn_prefill(x, x, x, scale=zero)
        with pytest.raises(ValueError, match="scale"):
            G.gdn_attn_decode(x, c, c, t, t[:, 0].contiguous(), scale=zero)


def test_the_reference_takes_a_scale_of_zero_as_it_is():
    rng = np.random.default_rng(0)
    q, k, v = (rng.standard_normal((5, 1, 4)) for _ in range(3))
    out, _, _ = A.attention(q, k, v, 0, scale=0.0)
    assert np.allclose(out[:, 0], [v[: i + 1, 0].mean(0) for i in range(5)])
    assert not np.allclose(A.attention(q, k, v, 0)[0], out)


@pytest.mark.parametrize("page", [2 ** 31, 2 ** 32 + 16, -2 ** 32 + 16, 2 ** 64])
def test_page_sizes_of_more_than_32_bits_are_refused(page):
    """2^32 + 16 must not pass for 16."""
    i, t = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: G.gdn_cache_plan(i, page, t, i, i[:1]), lambda: G.gdn_cache_release(i, i, page, t, i, i[:1])):
        with pytest.raises(ValueError, match="page_size"):
            call()


def test_a_scale_that_rounds_to_zero_is_refused():
    x = torch.randn(4, 2, 64)
    for tiny in (1e-46, -1e-300):
        with pytest.raises(ValueError, match="scale"):
            G.gdn_attn_prefill(x, x, x, scale=tiny)
    with pytest.raises(ValueError, match="GPU tensor"):
        G.gdn_attn_prefill(x, x, x, scale=1e-44)
