"""The operators around the projections together, as a recurrent layer runs
them, and in the settings a serving program puts them in: captured into
graphs, on side streams, from two threads, after each other on one
workspace (GPU)."""
import threading

import numpy as np
import pytest
import torch

import gated_deltanet_02_amd as G
from oracle import gates, layer
from tests import layer_util as U

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Layer:
    """A small recurrent layer: norm, projections, convolution, scan, gated
    norm, projection, on f32 so that one reference follows every step."""

    def __init__(self, seed, D=96, H=4, Gr=2, N=32, P=32):
        g = U.gen(seed)
        self.D, self.H, self.G, self.N, self.P, self.W = D, H, Gr, N, P, 4
        self.ch = H * P + 2 * Gr * N
        r = lambda *s: U.randn(g, *s)  # noqa: E731
        self.norm_w = 1 + 0.1 * r(D)
        self.w_in, self.w_dt, self.w_z = r(self.ch, D) / D ** 0.5, r(H, D) / D ** 0.5, r(H * P, D) / D ** 0.5
        self.w_out = r(D, H * P) / (H * P) ** 0.5
        self.taps, self.bias = r(self.ch, 4) / 2, 0.1 * r(self.ch)
        self.a_log = torch.log(1 + 15 * torch.rand(H, generator=g))
        self.dt_bias = -6.9 + 4.6 * torch.rand(H, generator=g)
        self.d_skip = 1 + 0.1 * r(H)
        self.gate_w = 1 + 0.1 * r(P)

    def cuda(self):
        c = object.__new__(Layer)
        c.__dict__.update({k: v.cuda() if torch.is_tensor(v) else v for k, v in self.__dict__.items()})
        return c

    def split(self, xbc):
        a, b = self.H * self.P, self.G * self.N
        t = xbc.shape[:-1]
        return (xbc[..., :a].unflatten(-1, (self.H, self.P)), xbc[..., a: a + b].unflatten(-1, (self.G, self.N)),
                xbc[..., a + b:].unflatten(-1, (self.G, self.N))) if t else None

    def prompt(self, x, res, cu, conv_state, state):
        y, res, _, _ = G.gdn_add_rms_norm(x, res, self.norm_w, residual_out=torch.empty_like(x))
        xbc = G.gdn_short_conv(y @ self.w_in.t(), self.taps, self.bias, cu_seqlens=cu, state_in=conv_state,
                               state_out=conv_state, silu=True)
        xs, b, c = self.split(xbc)
        o, _ = G.gdn_ssm_prefill(xs, y @ self.w_dt.t(), b, c, self.a_log, self.dt_bias, self.d_skip, cu, state,
                                 final_state=state)
        z = (y @ self.w_z.t()).view_as(o)
        return G.gdn_output_gate(o, z, self.gate_w).flatten(1) @ self.w_out.t(), res

    def step(self, x, res, conv_state, state):
        y, res, _, _ = G.gdn_add_rms_norm(x, res, self.norm_w, residual_out=torch.empty_like(x))
        xbc = G.gdn_short_conv((y @ self.w_in.t())[:, None], self.taps, self.bias, state_in=conv_state,
                               state_out=conv_state, silu=True)[:, 0]
        xs, b, c = self.split(xbc)
        o = G.gdn_ssm_decode(xs, y @ self.w_dt.t(), b, c, state, self.a_log, self.dt_bias, self.d_skip)
        z = (y @ self.w_z.t()).view_as(o)
        return G.gdn_output_gate(o, z, self.gate_w).flatten(1) @ self.w_out.t(), res

    def reference(self, x, res, lengths, conv_state, state):
        f = U.f64
        r, y, _ = layer.add_rms_norm(f(x), f(res), f(self.norm_w))
        xbc, conv_state, _ = layer.short_conv(y @ f(self.w_in).T, f(self.taps), f(self.bias), lengths, f(conv_state), True)
        T, a, b = x.shape[0], self.H * self.P, self.G * self.N
        xs, bb, cc = xbc[:, :a].reshape(T, self.H, self.P), xbc[:, a: a + b].reshape(T, self.G, self.N), xbc[:, a + b:].reshape(T, self.G, self.N)
        o, state = layer.ssm_scan(xs, y @ f(self.w_dt).T, bb, cc, f(self.a_log), f(self.dt_bias), f(self.d_skip), lengths, f(state))
        z = (y @ f(self.w_z).T).reshape(o.shape)
        o = gates.output_gate(o, z, f(self.gate_w), 1e-6)
        return o.reshape(T, -1) @ f(self.w_out).T, r, conv_state, state


def close(got, want, label):
    """f32 all through: each of the layer's six steps costs a few 2^-24 of
    sums of up to 128 terms; 2^-14 of the result's scale covers the chain."""
    got = U.f64(got)
    err = np.abs(got - want).max() / np.abs(want).max()
    print(f"  {label}: {err:.2e}", flush=True)
    assert err < 2.0 ** -14, label


def test_layer_prompts_then_steps():
    lengths, more = [70, 1, 0, 133], 6
    m = Layer(1)
    c = m.cuda()
    g = U.gen(2)
    n, T = len(lengths), sum(lengths)
    x, res = U.randn(g, T, m.D), 3 * U.randn(g, T, m.D)
    conv, st = U.randn(g, n, 3, m.ch), 0.5 * U.randn(g, n, m.H, m.N, m.P)
    gconv, gst = conv.cuda(), st.cuda()
    out, r = c.prompt(x.cuda(), res.cuda(), U.cu_of(lengths).cuda(), gconv, gst)
    want, wr, wconv, wst = m.reference(x, res, lengths, conv, st)
    for got, ref, label in ((out, want, "out"), (r, wr, "residual"), (gconv, wconv, "history"), (gst, wst, "state")):
        close(got, ref, "prompts " + label)
    for k in range(more):
        x, res = U.randn(g, n, m.D), U.randn(g, n, m.D)
        out, r = c.step(x.cuda(), res.cuda(), gconv, gst)
        want, wr, wconv, wst = m.reference(x, res, [1] * n, torch.from_numpy(wconv), torch.from_numpy(wst))
        for got, ref, label in ((out, want, "out"), (r, wr, "residual"), (gconv, wconv, "history"), (gst, wst, "state")):
            close(got, ref, f"step {k} {label}")


def scan_args(seed, T, n_seq, H=4, Gr=2, N=64, P=64):
    d = U.scan_inputs(seed, T, H, Gr, N, P, BF16, n_seq, init=True)
    return U.to_gpu(d)


def scan(e, cu, out, fin, ws, **kw):
    G.gdn_ssm_prefill(e["x"], e["dt"], e["b"], e["c"], e["a_log"], e["dt_bias"], e["d_skip"], cu, e["init"], out, fin,
                      segment_blocks=1, workspace=ws, **kw)


def test_captured_replays_follow_the_inputs():
    """One graph of every operator; inputs and lengths change between the
    replays, other work runs in between, every replay equals the eager run."""
    lengths = [[100, 40, 60], [1, 198, 1], [0, 0, 200], [67, 66, 67]]
    e = scan_args(1, 200, 3)
    cu = U.cu_of(lengths[0]).cuda()
    ws = G.ssm_workspace(e["x"], e["b"], cu, 1)
    out, fin = torch.empty_like(e["x"]), torch.empty_like(e["init"])
    taps, hist = torch.randn(256, 4, device="cuda"), torch.randn(3, 3, 256, device="cuda").to(BF16)
    new_hist = torch.empty_like(hist)
    conv_out = torch.empty(200, 256, dtype=BF16, device="cuda")
    res_out, q = torch.empty_like(conv_out), torch.empty(200, 256, device="cuda").to(torch.float8_e4m3fn)
    scales = torch.empty(200, 2, device="cuda")
    state, step_out = e["init"].clone(), torch.empty(3, 4, 64, dtype=BF16, device="cuda")

    def work():
        flat = e["x"].view(200, 256)
        G.gdn_short_conv(flat, taps, cu_seqlens=cu, state_in=hist, state_out=new_hist, silu=True, out=conv_out)
        G.gdn_add_rms_norm(conv_out, flat, residual_out=res_out, out_q=q, scales=scales)
        scan(e, cu, out, fin, ws)
        state.copy_(e["init"])
        G.gdn_ssm_decode(e["x"][:3], e["dt"][:3], e["b"][:3], e["c"][:3], state, e["a_log"], out=step_out)
        return [t.clone() for t in (conv_out, new_hist, res_out, q.float(), scales, out, fin, state, step_out)]

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = work()
    for k, ls in enumerate(lengths * 2):
        g = torch.Generator(device="cuda").manual_seed(k)
        for name in ("x", "b", "c", "dt", "init"):
            e[name].normal_(generator=g)
        hist.normal_(generator=g)
        cu.copy_(U.cu_of(ls))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        torch.randn(512, 512, device="cuda") @ torch.randn(512, 512, device="cuda")
        for i, (a, b) in enumerate(zip(got, work())):
            assert torch.equal(a, b), (k, i)


def test_side_stream_equals_current():
    e = scan_args(2, 300, 1)
    want = torch.empty_like(e["x"]), torch.empty_like(e["init"])
    ws = G.ssm_workspace(e["x"], e["b"], None, 1)
    scan(e, None, *want, ws)
    x = e["x"].view(300, 256)
    taps = torch.randn(256, 4, device="cuda")
    conv, norm = G.gdn_short_conv(x, taps), G.gdn_add_rms_norm(x)[0]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = torch.empty_like(e["x"]), torch.empty_like(e["init"])
    scan(e, None, *got, None, stream=s)  # its own workspace, from the stream's pool
    conv2 = G.gdn_short_conv(x, taps, stream=s)
    norm2 = G.gdn_add_rms_norm(x, stream=s)[0]
    # allocations on the current stream meanwhile
    junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(8)]
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(conv2, conv) and torch.equal(norm2, norm)
    del junk
    # by the raw handle
    out = G.gdn_short_conv(x, taps, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(out, conv)


def test_two_threads_on_their_own_streams():
    es = [scan_args(10 + i, 400, 1) for i in range(2)]
    want = []
    for e in es:
        o = torch.empty_like(e["x"]), torch.empty_like(e["init"])
        scan(e, None, *o, None)
        want.append(o)
    torch.cuda.synchronize()
    bad = []

    def run(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(10):
                    o = torch.empty_like(es[i]["x"]), torch.empty_like(es[i]["init"])
                    scan(es[i], None, *o, None)
                    s.synchronize()
                    if not (torch.equal(o[0], want[i][0]) and torch.equal(o[1], want[i][1])):
                        bad.append(i)
        except Exception as ex:  # noqa: BLE001
            bad.append(repr(ex))

    ts = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not bad


def test_calls_after_each_other_share_a_workspace():
    """Leftovers of a larger call do not reach a smaller one."""
    big, small = scan_args(3, 900, 1), scan_args(4, 130, 1)
    ws = G.ssm_workspace(big["x"], big["b"], None, 1)
    want = torch.empty_like(small["x"]), torch.empty_like(small["init"])
    scan(small, None, *want, None)
    ws.fill_(255)
    scan(big, None, torch.empty_like(big["x"]), torch.empty_like(big["init"]), ws)
    got = torch.empty_like(small["x"]), torch.empty_like(small["init"])
    scan(small, None, *got, ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_malformed_table_is_refused_under_the_debug_check(monkeypatch):
    monkeypatch.setenv("GDN_DEBUG_CHECK", "1")
    e = scan_args(5, 100, 2)
    x = e["x"].view(100, 256)
    bad = torch.tensor([0, 80, 60], dtype=torch.int32, device="cuda")
    with pytest.raises(G.GdnError) as ei:
        G.gdn_short_conv(x, torch.randn(256, 4, device="cuda"), cu_seqlens=bad)
    assert ei.value.status == -8
    with pytest.raises(G.GdnError) as ei:
        scan(e, bad, torch.empty_like(e["x"]), torch.empty_like(e["init"]), None)
    assert ei.value.status == -8


@pytest.mark.parametrize("n", [1500])
def test_many_sequences(n):
    """More sequences than the segment table's workgroup has threads, most of
    them of a few tokens, every tenth empty, some cut."""
    g = np.random.Generator(np.random.PCG64(7))
    lengths = [int(v) for v in g.integers(1, 6, n)]
    for i in range(0, n, 10):
        lengths[i] = 0
    lengths[5], lengths[1200] = 700, 500
    d = U.scan_inputs(6, sum(lengths), 2, 1, 16, 16, BF16, n, init=True)
    e = U.to_gpu(d)
    out, fin = torch.empty_like(e["x"]), torch.empty_like(e["init"])
    scan(e, U.cu_of(lengths, torch.int64).cuda(), out, fin, None)
    a = [U.f64(d[k]) for k in ("x", "dt", "b", "c", "a_log", "dt_bias", "d_skip")]
    y, s = layer.ssm_scan(*a, lengths=lengths, init=U.f64(d["init"]))
    my, ms = layer.ssm_magnitude(*a, lengths=lengths, init=U.f64(d["init"]))
    U.check(out, y, U.HALF[BF16] * np.abs(y) + U.SCAN_OUT * my, "many out")
    U.check(fin, s, U.SCAN_STATE * ms, "many states")
