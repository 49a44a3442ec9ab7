"""Strides that are never taken, of a single token, sequence or head, are any:
on the host, by the later refusal that such a call reaches, and on the GPU."""
import os

import numpy as np
import pytest
import torch

import gated_deltanet_02_amd as G
from gated_deltanet_02_amd import _binding as B
from gated_deltanet_02_amd import _layer as L
from oracle import layer
from tests import layer_util as U
from tests.test_layer_boundary import F32, I32, LAYOUT, WORKSPACE, expect, fake, message, scan, step

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.library_path()):
        pytest.fail("libgdn.so is not built (run __graft_entry__.build())")
    return L._functions()


def test_scan_of_one_token_or_head(lib):
    no_room = dict(ws=(None, 0), cu=fake((2,), I32))  # refused after the layout has been
    for kw in (dict(x=fake((1, 4, 32), strides=(1237, 32, 1))), dict(b=fake((1, 2, 64), strides=(131, 64, 1))),
               dict(c=fake((1, 2, 64), strides=(1 << 40, 64, 1))), dict(out=fake((1, 4, 32), strides=(7, 32, 1)))):
        expect(scan(lib, T=1, **kw, **no_room), WORKSPACE)
    for kw in (dict(x=fake((100, 1, 32), strides=(64, 13, 1))), dict(out=fake((100, 1, 32), strides=(32, 1, 1))),
               dict(b=fake((100, 1, 64), strides=(64, 3, 1))), dict(c=fake((100, 1, 64), strides=(128, 5, 1)))):
        expect(scan(lib, H=1, G=1, **kw, **no_room), WORKSPACE)
    # those that are taken, as before
    for kw in (dict(x=fake((2, 4, 32), strides=(1237, 32, 1))), dict(x=fake((2, 4, 32), strides=(1240, 33, 1)))):
        expect(scan(lib, T=2, **kw, **no_room), LAYOUT)


def test_step_of_one_sequence_or_head(lib):
    for n, H, strides in ((1, 4, (1237, 32, 1)), (3, 1, (64, 13, 1))):
        s = (n, H, 32)
        st = fake((n, H, 64, 32), F32)
        # an overlap, which is looked for after the strides
        expect(step(lib, n=n, H=H, G=1, x=fake(s, strides=strides), state=st, out=fake(s, addr=st.data)), LAYOUT)
        assert "overlaps" in message()
    expect(step(lib, n=2, x=fake((2, 4, 32), strides=(1237, 32, 1))), LAYOUT)
    assert "boundaries" in message()


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [1001, 1003])
def test_one_token_of_an_odd_projection(wide):
    """One row of a wider array of odd width, through the scan and the step."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    H, g, N, P = 4, 2, 32, 64
    d = U.scan_inputs(1, 1, H, g, N, P, BF16, 1, init=True)
    e = U.to_gpu(d)
    rows = torch.full((3, wide), float("nan"), dtype=BF16, device="cuda")
    flat = torch.cat([e["x"].flatten(), e["b"].flatten(), e["c"].flatten()])
    at = -(-wide // 8) * 8 - wide  # the second row's first 16-byte boundary
    rows[1, at: at + flat.numel()] = flat
    x, b, c = (v.view(1, *s) if v.numel() else v for v, s in zip(
        rows[1, at: at + flat.numel()].split([H * P, g * N, g * N]), [(H, P), (g, N), (g, N)]))
    x, b, c = (torch.as_strided(v, v.shape, (wide, v.stride(1), 1)) for v in (x, b, c))
    p = [e[k] for k in ("a_log", "dt_bias", "d_skip")]
    a = [U.f64(d[k]) for k in ("x", "dt", "b", "c", "a_log", "dt_bias", "d_skip")]
    y, s = layer.ssm_scan(*a, init=U.f64(d["init"]))
    my, ms = layer.ssm_magnitude(*a, init=U.f64(d["init"]))
    fin = torch.empty_like(e["init"])
    for cu in (None, U.cu_of([1]).cuda()):
        out, _ = G.gdn_ssm_prefill(x, e["dt"], b, c, *p, cu, e["init"], final_state=fin)
        U.check(out, y, U.HALF[BF16] * np.abs(y) + U.SCAN_OUT * my, "one token out")
        U.check(fin, s, U.SCAN_STATE * ms, "one token state")
    out = G.gdn_ssm_decode(x, e["dt"], b, c, e["init"], *p)
    U.check(out, y, U.HALF[BF16] * np.abs(y) + U.STEP_F32 * my, "one step out")
    U.check(e["init"], s, U.STEP_F32 * ms, "one step state")
