"""The residual norm over rows whose squares leave fp32's range (GPU): any
finite row has its norm, and without eps any row but zeros."""
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


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [3, 128, 1000, 4096, 20000])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_rows_of_every_size(dtype, D, eps):
    # values of 2^-120 to 2^120 a row, and rows of one large value among small ones
    size = torch.arange(-120, 121, 8 if D > 4096 else 1).float()
    x = torch.randn(len(size), D, generator=U.gen(D)).clamp(-4, 4) * torch.exp2(size)[:, None]
    x[::3, D // 2] *= 16
    x = x.to(dtype)
    for group in (0, 128):
        q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda")
        s = torch.empty((len(x), -(-D // 128)) if group else (len(x),), device="cuda")
        out, *_ = G.gdn_add_rms_norm(x.cuda(), None, None, eps, out=torch.empty_like(x, device="cuda"), out_q=q, scales=s)
        _, y, want = layer.add_rms_norm(U.f64(x), None, None, float(np.float32(eps)), group)
        # (below 2^-126 a step is no longer relative)
        U.check(out, y, (U.HALF[dtype] + U.NORM_F32) * np.abs(y) + 2.0 ** -126, f"D={D} {dtype} eps={eps}")
        U.check(s, want, U.NORM_F32 * want, "scales")
        per = np.repeat(want, group, axis=1)[:, :D] if group else want[:, None]
        U.check(U.f64(q) * per, y, np.maximum((2.0 ** -4 + 2.0 ** -14) * np.abs(y), 1.001 * 2.0 ** -10 * per), "codes")


def test_rows_of_infinities_and_zeros_as_before():
    x = torch.randn(4, 300, generator=U.gen(1))
    x[1, 7], x[2] = float("inf"), 0.0
    out, *_ = G.gdn_add_rms_norm(x.cuda(), None, None, 0.0)
    out = out.cpu()
    assert out[1, 7].isnan() and (out[1, :7] == 0).all() and (out[1, 8:] == 0).all()
    assert out[2].isnan().all() and out[0].isfinite().all() and out[3].isfinite().all()
