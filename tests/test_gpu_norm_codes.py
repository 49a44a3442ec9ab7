"""The residual norm's 8-bit codes, bit for bit (GPU): out_q is the fp32
quotient y / scales rounded to nearest even.  In fp32 ``out`` holds y itself,
so the quotient can be formed again here; PyTorch's division and conversion on
the CPU are the reference."""
import pytest
import torch

import gated_deltanet_02_amd as G
from tests import layer_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def rows(kind, R, D):
    g = U.gen(R + D)
    x = torch.randn(R, D, generator=g)
    if kind == "ties":
        # each 128 columns hold 448 k (the largest) and k times values half-way
        # between two codes
        at = torch.randint(0, 60, (R, D), generator=g)
        exp, odd = at // 8 - 3, at % 8
        x = (8.0 + odd + 0.5) * torch.exp2(exp.float()) * (1 - 2 * torch.randint(0, 2, (R, D), generator=g))
        x[:, ::128] = 448.0
    elif kind == "sizes":
        x = x * torch.exp2(torch.randint(-110, 60, (R, 1), generator=g).float())
    return x * (1 + torch.rand(R, 1, generator=g))


@pytest.mark.parametrize("kind", ["random", "ties", "sizes"])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("D", [1000, 256, 4096])
def test_codes_are_the_rounded_quotients(kind, group, D):
    R = 1024
    x = rows(kind, R, D)
    q = torch.empty(R, D, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((R, -(-D // group)) if group else (R,), device="cuda")
    # without eps the tiny rows are normed too
    out, *_ = G.gdn_add_rms_norm(x.cuda(), None, None, 0.0 if kind != "sizes" else 1e-6, out=torch.empty(R, D, device="cuda"),
                                 out_q=q, scales=s)
    y, s = out.cpu(), s.cpu()
    per = s.repeat_interleave(group, 1)[:, :D] if group else s[:, None]
    want = (y / per).to(torch.float8_e4m3fn)
    off = want.view(torch.uint8) != q.cpu().view(torch.uint8)
    print(f"  {kind} D={D} group={group}: {int(off.sum())} of {off.numel()} codes differ", flush=True)
    assert not off.any()


def test_infinite_weights_leave_the_other_columns_zero():
    """A scale of infinity: codes of zero for what is finite, NaN for what is
    not."""
    x = torch.randn(4, 256, generator=U.gen(1)).cuda()
    w = torch.ones(256, device="cuda")
    w[130] = float("inf")
    q, s = torch.empty(4, 256, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(4, 2, device="cuda")
    out, *_ = G.gdn_add_rms_norm(x, None, w, out=torch.empty_like(x), out_q=q, scales=s)
    f = q.float()
    assert s[:, 1].isinf().all() and s[:, 0].isfinite().all() and out[:, 130].isinf().all()
    assert f[:, 130].isnan().all() and (f[:, 128:130] == 0).all() and (f[:, 131:] == 0).all() and f[:, :128].isfinite().all()
