"""The selective state space scan and step against float64 (GPU)."""
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


def reference(d, lengths, act=True):
    a = [U.f64(d[k]) for k in ("x", "dt", "b", "c", "a_log", "dt_bias", "d_skip")]
    init = U.f64(d["init"])
    return (layer.ssm_scan(*a, lengths=lengths, init=init, act=act),
            layer.ssm_magnitude(*a, lengths=lengths, init=init, act=act))


def check_scan(d, out, final, lengths, label, act=True):
    (y, s), (my, ms) = reference(d, lengths, act)
    dtype = d["x"].dtype
    U.check(out, y, U.HALF[dtype] * np.abs(y) + U.SCAN_OUT * my, label + " out")
    if final is not None:
        U.check(final, s, U.SCAN_STATE * ms, label + " state")


def run(e, lengths, packed=True, **kw):
    cu = U.cu_of(lengths).cuda() if packed else None
    final = torch.full((len(lengths), e["x"].shape[1], e["b"].shape[2], e["x"].shape[2]), 7.0, device="cuda")
    out, fin = G.gdn_ssm_prefill(e["x"], e["dt"], e["b"], e["c"], e["a_log"], e["dt_bias"], e["d_skip"], cu, e["init"],
                                 final_state=final, **kw)
    return out, fin


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N", [16, 32, 64, 128])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_scan_sizes(dtype, N, P):
    """Every head size, ragged lengths around the block, a carried state."""
    lengths = [1, 63, 64, 65, 0, 130, 2]
    d = U.scan_inputs(N + P, sum(lengths), 4, 2, N, P, dtype, len(lengths), init=True)
    out, fin = run(U.to_gpu(d), lengths)
    check_scan(d, out, fin, lengths, f"scan N={N} P={P} {dtype}")


@pytest.mark.parametrize("n", [100, 128, 200, 256, 300, 512, 600])
@pytest.mark.parametrize("P", [32, 64])
def test_scan_many_sequences(n, P):
    """Numbers of segments around those at which their order changes (two
    heads, one or two workgroups a segment), lengths out of order, empty ones
    among them, one long enough to be cut."""
    lengths = [(37 * i * i + 11 * i) % 41 for i in range(n)]
    lengths[n // 3] = 300
    d = U.scan_inputs(n, sum(lengths), 2, 1, 32, P, BF16, n, init=True)
    e = U.to_gpu(d)
    for seg in (0, 1):
        out, fin = run(e, lengths, segment_blocks=seg)
        check_scan(d, out, fin, lengths, f"{n} sequences, segments {seg}")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("seg", [-1, 1, 2, 3])
@pytest.mark.parametrize("init", [True, False])
def test_scan_segments(dtype, seg, init):
    """Sequences cut into segments, beside short and empty ones."""
    lengths = [0, 700, 1, 0, 64, 129, 400, 0]
    d = U.scan_inputs(10 + seg, sum(lengths), 3, 1, 32, 64, dtype, len(lengths), init=init)
    out, fin = run(U.to_gpu(d), lengths, segment_blocks=seg)
    check_scan(d, out, fin, lengths, f"segments of {seg} {dtype}")


@pytest.mark.parametrize("B,L", [(1, 1), (1, 200), (2, 64), (3, 257), (5, 1)])
@pytest.mark.parametrize("seg", [0, 1])
def test_scan_batches(B, L, seg):
    d = U.scan_inputs(B + L, B * L, 2, 2, 64, 32, BF16, B, init=True)
    e = U.to_gpu(d)
    for k in ("x", "dt", "b", "c"):
        e[k] = e[k].view(B, L, *e[k].shape[1:])
    final = torch.empty_like(e["init"])
    out, fin = G.gdn_ssm_prefill(e["x"], e["dt"], e["b"], e["c"], e["a_log"], e["dt_bias"], e["d_skip"],
                                 init_state=e["init"], final_state=final, segment_blocks=seg)
    check_scan(d, out.view(B * L, 2, 32), fin, [L] * B, f"batch {B}x{L}")


@pytest.mark.parametrize("H,g", [(1, 1), (6, 6), (6, 3), (8, 1), (48, 16)])
def test_scan_groups(H, g):
    lengths = [90, 33]
    d = U.scan_inputs(H, sum(lengths), H, g, 64, 64, BF16, 2)
    out, fin = run(U.to_gpu(d), lengths)
    check_scan(d, out, fin, lengths, f"heads {H} groups {g}")


def test_scan_long_prompt():
    """2100 tokens, the automatic segments."""
    d = U.scan_inputs(1, 2100, 2, 1, 128, 128, BF16, 1, init=True)
    out, fin = run(U.to_gpu(d), [2100], packed=False)
    check_scan(d, out, fin, [2100], "long prompt")


def test_scan_without_parameters():
    """a_log, dt_bias and d_skip absent; dt as it is."""
    lengths = [70, 5]
    d = U.scan_inputs(2, 75, 2, 1, 32, 16, BF16, 2)
    d.update(dt=d["dt"].abs() * 0.1, a_log=None, dt_bias=None, d_skip=None)
    out, fin = run(U.to_gpu(d), lengths, softplus=False)
    check_scan(d, out, fin, lengths, "no parameters", act=False)


@pytest.mark.parametrize("kind", ["none", "strong", "mixed", "zero"])
def test_scan_decay_ranges(kind):
    """No decay at all, decays that underflow within a token, steps of zero."""
    lengths = [200, 64, 3]
    d = U.scan_inputs(3, sum(lengths), 2, 1, 64, 64, BF16, 3, init=True)
    if kind == "none":
        d["a_log"] = torch.full((2,), -40.0)
    elif kind == "strong":
        d["a_log"], d["dt_bias"] = torch.full((2,), 5.0), torch.full((2,), 3.0)
    elif kind == "mixed":
        d["dt"] = torch.where(torch.rand(d["dt"].shape, generator=U.gen(9)) < 0.3, torch.tensor(12.0), d["dt"])
    else:
        d["dt"] = torch.full_like(d["dt"], -200.0)
    out, fin = run(U.to_gpu(d), lengths, segment_blocks=1)
    check_scan(d, out, fin, lengths, f"decays {kind}")


def test_scan_column_views():
    """x, b and c as column ranges of one array, dt and out strided."""
    lengths = [100, 77]
    H, g, N, P = 4, 2, 32, 64
    d = U.scan_inputs(4, 177, H, g, N, P, BF16, 2)
    e = U.to_gpu(d)
    rows = torch.cat([e["x"].flatten(1), e["b"].flatten(1), e["c"].flatten(1)], 1).contiguous()
    e["x"] = rows[:, : H * P].view(177, H, P)
    e["b"] = rows[:, H * P: H * P + g * N].view(177, g, N)
    e["c"] = rows[:, H * P + g * N:].view(177, g, N)
    e["dt"] = e["dt"].t().contiguous().t()
    wide = torch.full((177, H, 2 * P), 3.0, dtype=BF16, device="cuda")
    out, fin = run(e, lengths, out=wide[:, :, :P])
    check_scan(d, out, fin, lengths, "column views")
    assert (wide[:, :, P:] == 3).all()


@pytest.mark.parametrize("seg", [-1, 1])
@pytest.mark.parametrize("packed", [True, False])
def test_scan_state_in_place(seg, packed):
    lengths = [500, 64, 0, 200] if packed else [400]
    d = U.scan_inputs(5, sum(lengths), 2, 1, 32, 32, BF16, len(lengths), init=True)
    e = U.to_gpu(d)
    state = e["init"].clone()
    out, fin = G.gdn_ssm_prefill(e["x"], e["dt"], e["b"], e["c"], e["a_log"], e["dt_bias"], e["d_skip"],
                                 U.cu_of(lengths).cuda() if packed else None, state, final_state=state,
                                 segment_blocks=seg)
    check_scan(d, out, fin, lengths, "state in place")


def test_scan_rows_past_the_batch_and_neighbours():
    """NaN after cu[N] and in one sequence reach nothing else; rows after
    cu[N] stay as they were."""
    lengths = [70, 20, 90]
    T = sum(lengths) + 30
    d = U.scan_inputs(6, T, 2, 1, 64, 64, BF16, 3, init=True)
    e = U.to_gpu(d)
    for k in ("x", "dt", "b", "c"):
        e[k] = e[k].clone()
        e[k][180:] = float("nan")
        e[k][70:90] = float("nan")
    out = torch.full_like(e["x"], 5.0)
    fin = torch.empty_like(e["init"])
    G.gdn_ssm_prefill(e["x"], e["dt"], e["b"], e["c"], e["a_log"], e["dt_bias"], e["d_skip"], U.cu_of(lengths).cuda(),
                      e["init"], out, fin, segment_blocks=1)
    assert (out[180:] == 5).all()
    parts = {k: v if k in ("a_log", "dt_bias", "d_skip") else v[[0, 2]] if k == "init" else torch.cat([v[:70], v[90:180]])
             for k, v in d.items()}
    check_scan(parts, torch.cat([out[:70], out[90:180]]), fin[[0, 2]], [70, 90], "neighbours")


def test_scan_malformed_table_stays_inside():
    e = U.to_gpu(U.scan_inputs(7, 128, 2, 1, 32, 32, BF16, 3))
    guard = torch.full((384, 2, 32), 9.0, dtype=BF16, device="cuda")
    for cu in ([0, 150, 20, 128], [5, -3, 400, 10], [0, 0, 0, 0], [128, 0, 128, 0]):
        G.gdn_ssm_prefill(e["x"], e["dt"], e["b"], e["c"], e["a_log"],
                          cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), out=guard[128:256],
                          segment_blocks=1)
    torch.cuda.synchronize()
    assert (guard[:128] == 9).all() and (guard[256:] == 9).all()


def test_scan_split_call_equals_whole():
    """A prompt in two calls, the state carried, against one call."""
    d = U.scan_inputs(8, 300, 2, 1, 64, 64, BF16, 1)
    e = U.to_gpu(d)
    args = lambda a, b: [e[k][a:b] for k in ("x", "dt", "b", "c")]  # noqa: E731
    p = [e[k] for k in ("a_log", "dt_bias", "d_skip")]
    st = torch.empty(1, 2, 64, 64, device="cuda")
    one, _ = G.gdn_ssm_prefill(*args(0, 111), *p, final_state=st)
    two, _ = G.gdn_ssm_prefill(*args(111, 300), *p, init_state=st, final_state=st)
    check_scan(d, torch.cat([one, two]), st, [300], "two calls")


def test_scan_repeats_bit_equal():
    d = U.scan_inputs(9, 1500, 3, 1, 128, 64, BF16, 1)
    e = U.to_gpu(d)
    first = run(e, [1500], packed=False)
    for _ in range(3):
        again = run(e, [1500], packed=False)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_scan_past_two_gib():
    """Element offsets past 2^31 in x and out."""
    H, P, N = 64, 128, 16
    T = (1 << 18) + 100
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(T, H, P, dtype=BF16, device="cuda").normal_(generator=g)
    b = torch.empty(T, 1, N, dtype=BF16, device="cuda").normal_(generator=g)
    c = torch.empty(T, 1, N, dtype=BF16, device="cuda").normal_(generator=g)
    dt = torch.empty(T, H, device="cuda").normal_(generator=g)
    n = 90
    cu = torch.tensor([0, T - n, T], device="cuda")
    out, _ = G.gdn_ssm_prefill(x, dt, b, c, cu_seqlens=cu)
    d = dict(x=x[-n:], dt=dt[-n:], b=b[-n:], c=c[-n:], a_log=None, dt_bias=None, d_skip=None, init=None)
    check_scan(d, out[-n:], None, [n], "far rows")


# ---------------------------------------------------------------------------
# the step


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N", [16, 32, 64, 128])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_step_sizes(dtype, N, P):
    n = 5
    d = U.scan_inputs(N * P, n, 6, 3, N, P, dtype, n, init=True)
    e = U.to_gpu(d)
    out = G.gdn_ssm_decode(e["x"], e["dt"], e["b"], e["c"], e["init"], e["a_log"], e["dt_bias"], e["d_skip"])
    (y, s), (my, ms) = reference(d, [1] * n)
    U.check(out, y, U.HALF[dtype] * np.abs(y) + U.STEP_F32 * my, f"step N={N} P={P}")
    U.check(e["init"], s, U.STEP_F32 * ms, f"step N={N} P={P} state")


@pytest.mark.parametrize("n,H,g", [(1, 1, 1), (1, 48, 16), (37, 4, 1)])
def test_step_views_and_defaults(n, H, g):
    N, P = 64, 32
    d = U.scan_inputs(n, n, H, g, N, P, BF16, n, init=True)
    d.update(a_log=None, dt_bias=None, d_skip=None, dt=d["dt"].abs())
    e = U.to_gpu(d)
    rows = torch.cat([e["x"].flatten(1), e["b"].flatten(1), e["c"].flatten(1)], 1).contiguous()
    x = rows[:, : H * P].view(n, H, P)
    b = rows[:, H * P: H * P + g * N].view(n, g, N)
    c = rows[:, H * P + g * N:].view(n, g, N)
    wide = torch.full((n, H, P + 4), 3.0, dtype=BF16, device="cuda")
    G.gdn_ssm_decode(x, e["dt"], b, c, e["init"], out=wide[:, :, :P], softplus=False)
    (y, s), (my, ms) = reference(d, [1] * n, act=False)
    U.check(wide[:, :, :P], y, U.HALF[BF16] * np.abs(y) + U.STEP_F32 * my, "step views")
    U.check(e["init"], s, U.STEP_F32 * ms, "step views state")
    assert (wide[:, :, P:] == 3).all()


def test_steps_follow_a_prompt():
    """A prompt's scan and then single tokens, against one longer scan."""
    n, L, more, H, N, P = 3, 90, 5, 2, 64, 64
    d = U.scan_inputs(11, n * (L + more), H, 1, N, P, F32, n)
    e = U.to_gpu(d)
    v = {k: e[k].view(n, L + more, *e[k].shape[1:]) for k in ("x", "dt", "b", "c")}
    p = [e[k] for k in ("a_log", "dt_bias", "d_skip")]
    st = torch.empty(n, H, N, P, device="cuda")
    outs = [G.gdn_ssm_prefill(*[v[k][:, :L].contiguous() for k in ("x", "dt", "b", "c")], *p, final_state=st)[0]]
    for t in range(L, L + more):
        outs.append(G.gdn_ssm_decode(*[v[k][:, t] for k in ("x", "dt", "b", "c")], st, *p)[:, None])
    check_scan(d, torch.cat(outs, 1).reshape(-1, H, P), st, [L + more] * n, "prompt and steps")


def test_step_state_past_two_gib():
    n, H, N, P = 1100, 16, 128, 128
    d = U.scan_inputs(12, n, H, 1, N, P, BF16, 1)
    e = U.to_gpu(d)
    g = torch.Generator(device="cuda").manual_seed(1)
    state = torch.empty(n, H, N, P, device="cuda").normal_(generator=g)
    last = state[-1:].clone()
    out = G.gdn_ssm_decode(e["x"], e["dt"], e["b"], e["c"], state, e["a_log"], e["dt_bias"], e["d_skip"])
    d1 = {k: v if k in ("a_log", "dt_bias", "d_skip", "init") else v[-1:] for k, v in d.items()}
    d1["init"] = last.cpu()
    (y, s), (my, ms) = reference(d1, [1])
    U.check(out[-1:], y, U.HALF[BF16] * np.abs(y) + U.STEP_F32 * my, "far step")
    U.check(state[-1:], s, U.STEP_F32 * ms, "far step state")


def test_step_of_more_sequences_than_one_launch():
    """2^32 threads and more: 64 of each 16 x 16 state (64 GiB of states)."""
    n, N = (1 << 26) + 5, 16
    g = torch.Generator(device="cuda").manual_seed(4)
    x, b, c = (torch.empty(n, 1, N, dtype=BF16, device="cuda").normal_(generator=g) for _ in range(3))
    dt = torch.rand(n, 1, generator=g, device="cuda")
    state = torch.zeros(n, 1, N, N, device="cuda")
    out = G.gdn_ssm_decode(x, dt, b, c, state, softplus=False)
    for rows in (slice(0, 3), slice((1 << 26) - 4, n)):
        d = dict(x=x[rows], dt=dt[rows], b=b[rows], c=c[rows], a_log=None, dt_bias=None, d_skip=None, init=None)
        k = rows.stop - rows.start
        (y, s), (my, ms) = reference(d, [1] * k, act=False)
        U.check(out[rows], y, U.HALF[BF16] * np.abs(y) + U.STEP_F32 * my, "step")
        U.check(state[rows], s, U.STEP_F32 * ms, "state")
    assert (out.float().abs().sum((1, 2)) > 0).float().mean() > 0.999
