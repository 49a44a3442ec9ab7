"""The operators around a recurrent layer's projections against float64
(GPU): the short convolution and the residual norm."""
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


# ---------------------------------------------------------------------------
# short convolution


def conv_case(seed, lengths, D, W, dtype, state=True, bias=True):
    g = U.gen(seed)
    d = dict(x=U.randn(g, sum(lengths), D, dtype=dtype), w=U.randn(g, D, W) / W ** 0.5,
             bias=0.1 * U.randn(g, D) if bias else None,
             hist=U.randn(g, len(lengths), W - 1, D, dtype=dtype) if state else None)
    return d, U.to_gpu(d)


def check_conv(d, out, state_out, lengths, silu, dtype, label):
    y, st, mag = layer.short_conv(U.f64(d["x"]), U.f64(d["w"]), U.f64(d["bias"]), lengths, U.f64(d["hist"]), silu)
    U.check(out, y, U.HALF[dtype] * np.abs(y) + U.CONV_F32 * (mag + 1), label)
    if state_out is not None:
        assert np.array_equal(U.f64(state_out), st), f"{label}: history"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("W", [1, 2, 3, 4])
@pytest.mark.parametrize("D", [8, 1, 37, 136, 1000])
def test_conv_packed(dtype, W, D):
    lengths = [1, 2, 0, 3, 17, 64, 5, 0, 31]
    d, e = conv_case(W * 100 + D, lengths, D, W, dtype)
    out = torch.full_like(e["x"], 7.0)
    st = torch.full_like(e["hist"], 7.0)
    for cu_type in (torch.int32, torch.int64):
        G.gdn_short_conv(e["x"], e["w"], e["bias"], cu_seqlens=U.cu_of(lengths, cu_type).cuda(), state_in=e["hist"],
                         state_out=st, silu=W % 2 == 0, out=out)
        check_conv(d, out, st, lengths, W % 2 == 0, dtype, f"conv D={D} W={W} {dtype}")


@pytest.mark.parametrize("shape", [(1, 1), (1, 5), (3, 1), (7, 2), (4, 33), (2, 300)])
@pytest.mark.parametrize("state", [True, False])
def test_conv_batches(shape, state):
    B, L = shape
    d, e = conv_case(B + L, [L] * B, 48, 4, BF16, state=state, bias=state)
    st = torch.empty(B, 3, 48, dtype=BF16, device="cuda")
    out = G.gdn_short_conv(e["x"].view(B, L, 48), e["w"], e["bias"], state_in=e["hist"], state_out=st, silu=True)
    assert out.shape == (B, L, 48)
    check_conv(d, out.view(B * L, 48), st, [L] * B, True, BF16, f"conv batch {shape}")


def test_conv_steps_equal_one_call():
    """Token by token with the history in place, bit-equal to the whole."""
    d, e = conv_case(3, [9] * 5, 64, 4, BF16)
    x = e["x"].view(5, 9, 64)
    whole = G.gdn_short_conv(x, e["w"], e["bias"], state_in=e["hist"], silu=True)
    state = e["hist"].clone()
    for t in range(9):
        step = G.gdn_short_conv(x[:, t: t + 1], e["w"], e["bias"], state_in=state, state_out=state, silu=True)
        assert torch.equal(step[:, 0], whole[:, t]), t
    assert torch.equal(state, x[:, 6:9])


@pytest.mark.parametrize("W", [2, 4])
def test_conv_in_place_history_of_short_and_long_sequences(W):
    lengths = [1, 40, 2, 0, 3, 100]
    d, e = conv_case(4, lengths, 72, W, F32)
    state = e["hist"].clone()
    out = G.gdn_short_conv(e["x"], e["w"], e["bias"], cu_seqlens=U.cu_of(lengths).cuda(), state_in=state, state_out=state)
    check_conv(d, out, state, lengths, False, F32, "conv in place")


@pytest.mark.parametrize("cols", [(0, 64, 96), (8, 64, 80), (3, 50, 61)])
def test_conv_strided_rows(cols):
    """Columns of a wider array, aligned for 16-byte accesses or not; what
    lies beside them stays as it was."""
    lo, n, wide = cols
    lengths = [5, 21]
    d, e = conv_case(5, lengths, n, 4, BF16)
    big = torch.full((26, wide), float("nan"), dtype=BF16, device="cuda")
    big[:, lo: lo + n] = e["x"]
    dst = torch.full((26, wide), 3.0, dtype=BF16, device="cuda")
    G.gdn_short_conv(big[:, lo: lo + n], e["w"], e["bias"], cu_seqlens=U.cu_of(lengths).cuda(), state_in=e["hist"],
                     out=dst[:, lo: lo + n])
    check_conv(d, dst[:, lo: lo + n], None, lengths, False, BF16, f"conv columns {cols}")
    assert (dst[:, :lo] == 3).all() and (dst[:, lo + n:] == 3).all()


def test_conv_rows_past_the_batch_and_neighbours():
    """Rows at or after cu[N] (NaN) are neither read into results nor
    written; a sequence of NaN leaves its neighbours finite."""
    lengths = [20, 3, 33]
    d, e = conv_case(6, lengths + [11], 40, 4, F32)
    x = e["x"].clone()
    x[56:] = float("nan")
    x[20:23] = float("nan")
    out = torch.full_like(x, 5.0)
    G.gdn_short_conv(x, e["w"], e["bias"], cu_seqlens=U.cu_of(lengths).cuda(), state_in=e["hist"][:3], out=out)
    y = layer.short_conv(U.f64(d["x"]), U.f64(d["w"]), U.f64(d["bias"]), lengths + [11], U.f64(d["hist"]))
    keep = [*range(20), *range(23, 56)]
    U.check(out[keep], y[0][keep], U.HALF[F32] * np.abs(y[0][keep]) + U.CONV_F32 * (y[2][keep] + 1), "conv neighbours")
    assert (out[56:] == 5).all()


def test_conv_malformed_table_stays_inside():
    """Decreasing and out-of-range entries give some output without touching
    anything beside the tensors."""
    x = torch.randn(64, 32, device="cuda")
    guard = torch.full((64 * 3, 32), 9.0, device="cuda")
    w = torch.randn(32, 4, device="cuda")
    for cu in ([0, 70, 20, 64], [5, -3, 400, 10], [0, 0, 0, 0], [64, 0, 64, 0]):
        G.gdn_short_conv(x, w, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), out=guard[64:128])
    torch.cuda.synchronize()
    assert (guard[:64] == 9).all() and (guard[128:] == 9).all()


def test_conv_past_two_gib():
    """Element offsets past 2^31."""
    D, T = 4096, (1 << 19) + 40
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(T, D, dtype=BF16, device="cuda").normal_(generator=g)
    w = torch.randn(D, 4, generator=g, device="cuda")
    out = G.gdn_short_conv(x, w)
    tail = x[-24:].double().cpu().numpy()
    y, _, mag = layer.short_conv(tail, U.f64(w))
    U.check(out[-20:], y[4:], U.HALF[BF16] * np.abs(y[4:]) + U.CONV_F32 * (mag[4:] + 1), "conv far rows")


# ---------------------------------------------------------------------------
# residual norm


def norm_case(seed, R, D, dtype, residual=True, weight=True):
    g = U.gen(seed)
    d = dict(x=U.randn(g, R, D, dtype=dtype),
             residual=(U.randn(g, R, D) * torch.exp(2 * U.randn(g, R, 1))).to(dtype) if residual else None,
             weight=1 + 0.1 * U.randn(g, D) if weight else None)
    return d, U.to_gpu(d)


def check_norm(d, got, group, label):
    dtype = d["x"].dtype
    r, y, s = layer.add_rms_norm(U.f64(d["x"]), U.f64(d["residual"]), U.f64(d["weight"]), 1e-6, group)
    if got.get("residual_out") is not None:
        U.check(got["residual_out"], r, (U.HALF[dtype] + 2.0 ** -23) * np.abs(r), label + " residual")
    if got.get("out") is not None:
        U.check(got["out"], y, (U.HALF[dtype] + U.NORM_F32) * np.abs(y), label + " out")
    if got.get("out_q") is not None:
        U.check(got["scales"], s, U.NORM_F32 * s, label + " scales")
        per = np.repeat(s, group, axis=1)[:, : y.shape[1]] if group else s[:, None]
        mine = U.f64(got["scales"])
        mine = np.repeat(mine, group, axis=1)[:, : y.shape[1]] if group else mine[:, None]
        # half a step relative, or half the smallest step (2^-9) near zero
        bound = np.maximum((U.HALF[torch.float8_e4m3fn] + 2.0 ** -14) * np.abs(y), 1.001 * 2.0 ** -10 * per)
        U.check(U.f64(got["out_q"]) * mine, y, bound, label + " 8 bits")


def norm_outputs(x, which, group):
    R, D = x.shape
    got = {}
    if "r" in which:
        got["residual_out"] = torch.empty_like(x)
    if "y" in which:
        got["out"] = torch.empty_like(x)
    if "q" in which:
        got["out_q"] = torch.empty(R, D, dtype=torch.float8_e4m3fn, device="cuda")
        got["scales"] = torch.empty((R, -(-D // group)) if group else (R,), device="cuda")
    return got


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [1, 7, 8, 64, 100, 128, 136, 512, 520, 1024, 1032, 2048, 2500, 4096, 5120, 6144, 8192, 8200,
                               16384, 20000, 65536])
@pytest.mark.parametrize("group", [0, 128])
def test_norm_widths(dtype, D, group):
    R = 5
    d, e = norm_case(D, R, D, dtype)
    got = norm_outputs(e["x"], "ryq", group)
    G.gdn_add_rms_norm(e["x"], e["residual"], e["weight"], **got)
    check_norm(d, got, group, f"norm D={D} group={group} {dtype}")


@pytest.mark.parametrize("which", ["r", "y", "q", "ry", "rq", "yq"])
@pytest.mark.parametrize("R", [1, 4, 131])
def test_norm_outputs(which, R):
    d, e = norm_case(R, R, 384, BF16, residual="r" in which, weight=R != 4)
    got = norm_outputs(e["x"], which, 0)
    G.gdn_add_rms_norm(e["x"], e["residual"], e["weight"], **got)
    check_norm(d, got, 0, f"norm {which} R={R}")


def test_norm_default_output():
    d, e = norm_case(1, 3, 96, F32, residual=False, weight=False)
    out, ro, q, s = G.gdn_add_rms_norm(e["x"])
    assert ro is None and q is None and s is None
    check_norm(d, {"out": out}, 0, "norm default")


@pytest.mark.parametrize("D", [256, 250])
def test_norm_in_place(D):
    """residual_out over the residual and out over x; also over x."""
    d, e = norm_case(2, 9, D, BF16)
    x, r = e["x"].clone(), e["residual"].clone()
    G.gdn_add_rms_norm(x, r, e["weight"], residual_out=r, out=x)
    check_norm(d, {"residual_out": r, "out": x}, 0, "norm in place")
    x = e["x"].clone()
    out = G.gdn_add_rms_norm(x, e["residual"], e["weight"], residual_out=x, out=torch.empty_like(x))[0]
    check_norm(d, {"residual_out": x, "out": out}, 0, "norm over x")


@pytest.mark.parametrize("cols", [(0, 256, 320), (8, 136, 160), (5, 99, 120)])
def test_norm_strided_rows(cols):
    lo, n, wide = cols
    d, e = norm_case(7, 6, n, BF16)
    big = torch.full((6, wide), float("nan"), dtype=BF16, device="cuda")
    big[:, lo: lo + n] = e["x"]
    dst = torch.full((6, wide), 3.0, dtype=BF16, device="cuda")
    dq = torch.full((6, wide), 3.0, device="cuda").to(torch.float8_e4m3fn)
    got = {"out": dst[:, lo: lo + n], "out_q": dq[:, lo: lo + n], "scales": torch.empty(6, -(-n // 128), device="cuda")}
    G.gdn_add_rms_norm(big[:, lo: lo + n], e["residual"], e["weight"], **got)
    check_norm(d, got, 128, f"norm columns {cols}")
    for v in (dst, dq.float()):
        assert (v[:, :lo] == 3).all() and (v[:, lo + n:] == 3).all()


def test_norm_zero_tiny_and_large_rows():
    """Rows of zeros, rows whose squares underflow or are large, and single
    spikes: scales stay finite and no value leaves the 8-bit range."""
    x = torch.zeros(6, 256)
    x[1] = 1e-25
    x[2] = 1e15 * torch.randn(256, generator=U.gen(1))
    x[3, 17] = 5.0
    x[4] = -2.0
    x[5, :128] = torch.randn(128, generator=U.gen(2))
    d = dict(x=x, residual=None, weight=None)
    for group in (0, 128):
        e = U.to_gpu(d)
        got = norm_outputs(e["x"], "yq", group)
        G.gdn_add_rms_norm(e["x"], None, None, **got)
        check_norm(d, got, group, f"norm rows group={group}")


def test_norm_nan_rows_stay_rows():
    d, e = norm_case(8, 5, 512, F32)
    x = e["x"].clone()
    x[2, 300] = float("nan")
    for group in (0, 128):
        got = norm_outputs(x, "yq", group)
        G.gdn_add_rms_norm(x, e["residual"], e["weight"], **got)
        assert got["out"][2].isnan().all() and got["scales"][2].isnan().all()
        assert got["out_q"][2].float().isnan().all()
        keep = [0, 1, 3, 4]
        check_norm({k: v[keep] if k != "weight" else v for k, v in d.items()}, {k: v[keep] for k, v in got.items()}, group,
                   "norm beside a NaN row")


def test_norm_no_rows():
    x = torch.empty(0, 64, device="cuda")
    out, *_ = G.gdn_add_rms_norm(x)
    assert out.shape == (0, 64)


def test_norm_past_two_gib():
    R, D = 70000, 32768
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(R, D, dtype=BF16, device="cuda").normal_(generator=g)
    q = torch.empty(R, D, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(R, 256, device="cuda")
    out, *_ = G.gdn_add_rms_norm(x, out=torch.empty_like(x), out_q=q, scales=s)
    check_norm(dict(x=x[-2:], residual=None, weight=None), {"out": out[-2:], "out_q": q[-2:], "scales": s[-2:]}, 128,
               "norm far rows")


@pytest.mark.parametrize("dtype,group", [(BF16, 0), (F32, 128)])
def test_norm_more_rows_than_one_launch(dtype, group):
    """Rows around 2^21, where the library starts another launch."""
    R, D, at = (1 << 21) + 7, 40, 1 << 21
    g = torch.Generator(device="cuda").manual_seed(3)
    big = torch.empty(R, 48, dtype=dtype, device="cuda").normal_(generator=g)
    x, res = big[:, :D], torch.empty(R, D, dtype=dtype, device="cuda").normal_(generator=g)
    w = torch.rand(D, generator=g, device="cuda")
    q = torch.zeros(R, D, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.zeros((R, 1) if group else (R,), device="cuda")
    out, ro, *_ = G.gdn_add_rms_norm(x, res, w, residual_out=torch.zeros_like(res), out=torch.zeros_like(res),
                                     out_q=q, scales=s)
    for rows in (slice(0, 5), slice(at - 5, at + 5), slice(R - 3, R)):
        check_norm(dict(x=x[rows], residual=res[rows], weight=w),
                   {"out": out[rows], "residual_out": ro[rows], "out_q": q[rows], "scales": s[rows]}, group,
                   f"rows {rows.start}")
    assert (s > 0).all() and (out.float().abs().sum(1) > 0).all()
