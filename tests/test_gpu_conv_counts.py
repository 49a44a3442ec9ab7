"""The short convolution at counts past what a launch or a 32-bit sum of two
indices holds (GPU)."""
import time

import numpy as np
import pytest
import torch

import gated_deltanet_02_amd as G
from oracle import layer
from tests import layer_util as U

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def far_apart(n, lengths, dtype, W=3):
    """Sequences 0 .. n - 1 with the given lengths at some indices, the rest
    empty, one channel, against float64."""
    cu = torch.zeros(n + 1, dtype=dtype, device="cuda")
    for i, length in lengths.items():
        cu[i + 1:] += length
    T = sum(lengths.values())
    g = U.gen(1)
    x, w, bias = U.randn(g, T, 1), U.randn(g, 1, W), U.randn(g, 1)
    d = U.to_gpu(dict(x=x, w=w, bias=bias))
    out = torch.full((T, 1), 7.0, device="cuda")
    torch.cuda.synchronize()
    began = time.monotonic()
    G.gdn_short_conv(d["x"], d["w"], d["bias"], cu_seqlens=cu, out=out)
    torch.cuda.synchronize()
    took = time.monotonic() - began
    y, _, mag = layer.short_conv(U.f64(x), U.f64(w), U.f64(bias), [lengths[i] for i in sorted(lengths)])
    U.check(out, y, U.HALF[F32] * np.abs(y) + U.CONV_F32 * (mag + 1), f"{n} sequences, {took:.3f} s")
    return took


def test_long_runs_of_empty_sequences():
    """Are passed over, not walked through: 2^24 of them one by one are that
    many loads in a row, some seconds."""
    n = 1 << 24
    assert far_apart(n, {0: 50, 2: 3, n // 2: 70, n // 2 + 1: 1, n - 1: 33}, torch.int32) < 1.0


@pytest.mark.parametrize("cu_type", [torch.int32, torch.int64])
def test_more_than_two_to_the_thirty_sequences(cu_type):
    """Nearly all of them empty; those with tokens lie at both ends, so that
    the search for a token's sequence adds indices whose sum passes 2^31."""
    n = (1 << 30) + 9
    far_apart(n, {0: 50, 2: 3, n - 9: 70, n - 3: 1, n - 1: 33}, cu_type)


@pytest.mark.parametrize("packed", [False, True])
def test_more_steps_than_one_launch(packed):
    """2^24 workgroups and more: one token for each of 8.4 million sequences,
    the histories in place, each read and written once."""
    D, W, split = 257, 2, 8388604  # two workgroups a sequence
    n = split + 50
    g = torch.Generator(device="cuda").manual_seed(2)
    x, state = (torch.empty(n, D, dtype=BF16, device="cuda").normal_(generator=g) for _ in range(2))
    w, bias = torch.randn(D, W, generator=g, device="cuda"), torch.randn(D, generator=g, device="cuda")
    rows = [slice(0, 4), slice(split // 2, split // 2 + 4), slice(split - 8, split + 8), slice(n - 4, n)]
    before = [state[r].clone() for r in rows]
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda") if packed else None
    out = torch.zeros(n, D, dtype=BF16, device="cuda")
    G.gdn_short_conv(x if packed else x[:, None], w, bias, cu_seqlens=cu, state_in=state[:, None],
                     state_out=state[:, None], out=out if packed else out[:, None])
    assert torch.equal(state, x)
    for r, old in zip(rows, before):
        k = r.stop - r.start
        y, _, mag = layer.short_conv(U.f64(x[r]), U.f64(w), U.f64(bias), [1] * k, U.f64(old[:, None]))
        U.check(out[r], y, U.HALF[BF16] * np.abs(y) + U.CONV_F32 * (mag + 1), f"rows from {r.start}")
