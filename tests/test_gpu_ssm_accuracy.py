"""How exact the state space scan is, token by token, beside 64 bits (GPU):
fp32 inputs against bounds of their own, and decays of every size in both
types.

Bounds for fp32 inputs.  Everything is then formed in fp32, each rounding at
most 2^-24.  A sum of n terms of like size and random sign rounds n times at
the size of its partial sums: together sqrt(n / 2) 2^-24 of the result's size.
An output passes through three such sums, c.b and S^T c over N <= 128 (8 each)
and M x over 32 tokens (4), and a state through the 32 tokens of each block
(4) and one more rounding a block (at most 6 for 64 blocks without decay); a
step, its decay and their exponent carry about 4 roundings that a token's
products share.  sqrt(8^2 + 8^2 + 4^2 + 4^2) < 13 and 13 2^-24 < 2^-20: the
root mean square, over tokens and heads, of an output vector's relative
error, and of a head's state likewise, stays below 2^-20 (one output in two
bf16 terms would reach 2^-19).  No single vector is further off than 2^-19 of
the same sums over absolute values.

A decay e^-x from an exponent that is rounded (d, the rate and their product:
four roundings) is x 4 2^-24 off.  Steps up to 1 keep x e^-x below 0.4 and add
nothing to the above; what a step of s leaves behind is still of the size of
the rest where it has decayed by 1 / s, and adds ln(s) 2^-22 to both bounds.

Two sizes that a relative error cannot be taken of.  fp32 ends at 2^-126, so a
memory decayed by e^-300 has to come out as 0: vectors below 2^-100 count as
of that size.  And behind a token whose step d ends all memory, out = (D +
d c.b) x is one number times x: where that number nearly vanishes, its terms
still round at their own sizes.  N = 32 products of random sign come to
0.28 of their absolute sum in the root mean square (sqrt(32) against 32
(2 / pi)) and to less than 1/16 of it in one of six; those count as 1/16.
"""
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


def check_vectors(got, want, mag, axes, label, step):
    """The two bounds above; a vector is what ``axes`` span, ``step`` the largest
    step."""
    more = np.log(max(step, 1.0)) * 2.0 ** -22
    got = U.f64(got)
    assert np.isfinite(got).all(), f"{label}: not finite"
    norm = lambda v: np.sqrt((np.asarray(v) ** 2).sum(axes))  # noqa: E731
    err, size, most = norm(got - want), norm(want), norm(mag)
    rms = float(np.sqrt(np.mean((err / np.maximum(np.maximum(size, most / 16), 2.0 ** -100)) ** 2)))
    worst = float((err / np.maximum(most, 2.0 ** -100)).max())
    print(f"  {label}: rms {rms:.2e}, worst {worst:.2e} of the absolute sums", flush=True)
    assert rms <= 2.0 ** -20 + more, label
    assert worst <= 2.0 ** -19 + more, label


def check(d, lengths, label, step=1.0, **kw):
    e = U.to_gpu(d)
    fin = torch.empty(len(lengths), e["x"].shape[1], e["b"].shape[2], e["x"].shape[2], device="cuda")
    out, _ = G.gdn_ssm_prefill(e["x"], e["dt"], e["b"], e["c"], e["a_log"], e["dt_bias"], e["d_skip"],
                               U.cu_of(lengths).cuda(), e["init"], final_state=fin, **kw)
    a = [U.f64(d[k]) for k in ("x", "dt", "b", "c", "a_log", "dt_bias", "d_skip")]
    y, s = layer.ssm_scan(*a, lengths=lengths, init=U.f64(d["init"]))
    my, ms = layer.ssm_magnitude(*a, lengths=lengths, init=U.f64(d["init"]))
    if d["x"].dtype == F32:
        check_vectors(out, y, my, 2, label + " out", step)
        check_vectors(fin, s, ms, (2, 3), label + " state", step)
    else:
        U.check(out, y, U.HALF[BF16] * np.abs(y) + U.SCAN_OUT * my + 2.0 ** -100, label + " out")
        U.check(fin, s, U.SCAN_STATE * ms + 2.0 ** -100, label + " state")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rate", [1.0, 16.0, 148.0])
@pytest.mark.parametrize("step", [2.0, 20.0, 100.0, 1000.0, 1e6, 1e30])
def test_large_steps_among_small_ones(dtype, rate, step):
    """Single tokens whose step ends all memory, at every place of a tile of
    16, among ordinary ones: what follows them is as exact as anything else.
    Half of them carry nothing of their own, so that the tokens behind them
    are seen."""
    lengths = [16 * 17 + 5, 40]
    T, H = sum(lengths), 2
    d = U.scan_inputs(int(step) % 97 + int(rate), T, H, 1, 32, 64, dtype, 2, init=True)
    d["a_log"] = torch.full((H,), rate).log()
    d["dt_bias"] = torch.full((H,), -4.0)
    at = torch.arange(0, T, 17)  # 0, 1, 2, ... of their tiles
    d["dt"][at] = step + 4.0
    d["dt"][at[::3] + 2] = step + 4.0  # a second one two tokens on
    d["x"][at[::2]] = 0.0
    for seg in (-1, 1):
        check(d, lengths, f"rate {rate} step {step} {dtype} segments {seg}", step, segment_blocks=seg)


@pytest.mark.parametrize("N", [16, 32, 64, 128])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_fp32_sizes(N, P):
    """Every head size, ragged lengths around the blocks, one cut."""
    lengths = [1, 63, 64, 65, 0, 130, 2]
    d = U.scan_inputs(N + 3 * P, sum(lengths), 4, 2, N, P, F32, len(lengths), init=True)
    for seg in (-1, 1):
        check(d, lengths, f"N={N} P={P} segments {seg}", segment_blocks=seg)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ["none", "strong", "mixed", "zero", "large"])
@pytest.mark.parametrize("rate", [1.0, 16.0, 148.0])
def test_decay_ranges_and_rates(dtype, kind, rate):
    """No memory lost, lost within a token, now and then, with steps of zero
    and of some hundred, at every rate."""
    lengths = [200, 64, 3]
    d = U.scan_inputs(3, sum(lengths), 2, 1, 64, 64, dtype, 3, init=True)
    d["a_log"] = torch.full((2,), -40.0) if kind == "none" else torch.full((2,), rate).log()
    step = 1.0
    if kind == "strong":
        d["dt_bias"], step = torch.full((2,), 3.0), 8.0
    elif kind == "mixed":
        d["dt"] = torch.where(torch.rand(d["dt"].shape, generator=U.gen(9)) < 0.3, torch.tensor(12.0), d["dt"])
        step = 12.0
    elif kind == "zero":
        d["dt"] = torch.full_like(d["dt"], -200.0)
    elif kind == "large":
        d["dt"], step = 100 + 100 * d["dt"].abs(), 600.0
    for seg in (-1, 1):
        check(d, lengths, f"{kind} rate {rate} {dtype} segments {seg}", step, segment_blocks=seg)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rates_past_the_largest_float(dtype):
    """e^a_log beyond fp32: any step ends all memory, a step of zero none; in
    the scan and in the step."""
    lengths, H = [45, 20], 2
    d = U.scan_inputs(7, sum(lengths), H, 1, 32, 32, dtype, 2, init=True)
    d["a_log"] = torch.tensor([100.0, 88.6])
    d["dt"][::3] = -200.0
    for seg in (-1, 1):
        check(d, lengths, f"rates past the largest {dtype} segments {seg}", segment_blocks=seg)
    d = U.scan_inputs(8, 6, H, 1, 32, 32, F32, 6, init=True)
    d["a_log"] = torch.tensor([100.0, 88.6])
    d["dt"][::2] = -200.0
    e = U.to_gpu(d)
    out = G.gdn_ssm_decode(e["x"], e["dt"], e["b"], e["c"], e["init"], e["a_log"], e["dt_bias"], e["d_skip"])
    a = [U.f64(d[k]) for k in ("x", "dt", "b", "c", "a_log", "dt_bias", "d_skip")]
    y, s = layer.ssm_scan(*a, lengths=[1] * 6, init=U.f64(d["init"]))
    my, ms = layer.ssm_magnitude(*a, lengths=[1] * 6, init=U.f64(d["init"]))
    check_vectors(out, y, my, 2, "step out", 1.0)
    check_vectors(e["init"], s, ms, (2, 3), "step state", 1.0)
