"""The recurrent layer's operators around the projections, as measured cases: the short causal convolution, the selective state space scan (prompts and single tokens), and the
root-mean-square norm with the residual's addition and an 8-bit output.  Each is computed either in its plain form (elementary torch operations in float32, decays and their sums in
float64) or by the library's entry points."""
import math

import torch

own = False

E4M3_MAX = 448.0
SCALE_FLOOR = 2.0 ** -100
GROUP = 128
CHUNK = 64  # tokens per block of the plain scan


def _prompts(count, low, high, seed):
    """Prompt lengths of a packed batch, spread evenly over [low, high] in an order that the seed shuffles: the total does not depend on the seed."""
    lengths = torch.linspace(low, high, count).round().to(torch.int64)
    return lengths[torch.randperm(count, generator=torch.Generator().manual_seed(seed))].tolist()


def _lengths(case, seed):
    if case["lengths"] == "spread":
        return _prompts(case["seqs"], case["low"], case["high"], seed)
    return [int(v) for v in case["lengths"].split(",")]


def listed():
    conv = {"op": "conv", "dtype": "bf16", "width": 4, "silu": True}
    scan = {"op": "scan", "dtype": "bf16", "init": False}
    step = {"op": "step", "dtype": "bf16"}
    norm = {"op": "norm", "dtype": "bf16", "residual": True, "out": True, "scales": "none"}
    return [
        # one token for each of 256 running sequences, the channels of 16 heads of 128 with 16 groups of 128
        {"name": "conv step", **conv, "lengths": ",".join(["1"] * 256), "channels": 6144},
        # a packed batch of prompts
        {"name": "conv prompts", **conv, "lengths": "spread", "seqs": 64, "low": 200, "high": 4096, "channels": 6144},
        # channels that no vector access fits, three taps, no activation
        {"name": "conv odd", **conv, "dtype": "f32", "width": 3, "silu": False, "lengths": "1000,1,2,234", "channels": 1001},
        # one prompt at the default length limit
        {"name": "scan prompt", **scan, "lengths": "4096", "heads": 16, "groups": 16, "n": 128, "p": 128},
        # the longest prompt, three heads to a group, continuing a carried state
        {"name": "scan long", **scan, "lengths": "16384", "heads": 48, "groups": 16, "n": 128, "p": 128, "init": True},
        # a packed batch of prompts, small heads sharing two groups
        {"name": "scan prompts", **scan, "lengths": "spread", "seqs": 64, "low": 200, "high": 4096, "heads": 16, "groups": 2, "n": 128, "p": 64},
        # ragged lengths around the block size, float32
        {"name": "scan edge", **scan, "dtype": "f32", "lengths": "1,63,64,65,1000", "heads": 8, "groups": 8, "n": 64, "p": 32, "init": True},
        # one token for each of 256 running sequences
        {"name": "step 256", **step, "seqs": 256, "heads": 16, "groups": 16, "n": 128, "p": 128},
        # a single running sequence
        {"name": "step 1", **step, "seqs": 1, "heads": 48, "groups": 16, "n": 128, "p": 128},
        # a prompt's rows before the projections, in 8 bits with a scale for each row
        {"name": "norm prompt", **norm, "rows": 4096, "width": 5120, "scales": "row"},
        # a few running sequences
        {"name": "norm step", **norm, "rows": 8, "width": 4096},
        # a packed batch of prompts, 8 bits alone, scales for each 128 columns
        {"name": "norm prompts", **norm, "rows": 131071, "width": 6144, "out": False, "scales": "group"},
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["conv", "scan", "step", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "conv":
        channels = _log_int(rng, 17, 6144)
        if rng.random() < 0.7:
            channels = max(8, channels // 8 * 8)
        case = {"op": op, "dtype": dtype, "width": rng.randint(2, 4), "silu": rng.random() < 0.7, "channels": channels}
        return {**case, **_draw_lengths(rng, 65536)}
    if op == "scan":
        groups = rng.choice([1, 2, 4, 8])
        heads = groups * rng.choice([1, 2, 3, 4])
        case = {"op": op, "dtype": dtype, "init": rng.random() < 0.5, "heads": heads, "groups": groups, "n": rng.choice([16, 32, 64, 128]), "p": rng.choice([16, 32, 64, 128])}
        return {**case, **_draw_lengths(rng, 32768)}
    if op == "step":
        groups = rng.choice([1, 2, 4, 8, 16])
        return {"op": op, "dtype": dtype, "seqs": _log_int(rng, 1, 256), "heads": groups * rng.choice([1, 2, 3]), "groups": groups, "n": rng.choice([16, 32, 64, 128]), "p": rng.choice([16, 32, 64, 128])}
    width = _log_int(rng, 33, 16384)
    if rng.random() < 0.7:
        width = max(8, width // 8 * 8)
    rows = _log_int(rng, 1, max(1, min(65536, (1 << 28) // width)))
    scales = rng.choice(["none", "row", "group"])
    return {"op": op, "dtype": dtype, "rows": rows, "width": width, "residual": rng.random() < 0.7, "out": scales == "none" or rng.random() < 0.5, "scales": scales}


def _draw_lengths(rng, most):
    """One prompt, a few ragged ones (an empty one among them now and then), or a spread of many."""
    kind = rng.random()
    if kind < 0.4:
        return {"lengths": str(_log_int(rng, 1, min(16384, most)))}
    if kind < 0.8:
        lengths = [_log_int(rng, 1, 4096) for _ in range(rng.randint(2, 8))]
        if rng.random() < 0.3:
            lengths[rng.randrange(len(lengths))] = 0
        return {"lengths": ",".join(str(v) for v in lengths)}
    seqs = rng.randint(9, max(9, most // 2148))
    return {"lengths": "spread", "seqs": seqs, "low": 200, "high": 4096}


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


class _Draws:
    """Seeded draws on the GPU."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(self, *shape, dtype=torch.float32):
        return torch.randn(*shape, generator=self.g, device="cuda", dtype=dtype)

    def uniform(self, low, high, *shape):
        return torch.rand(*shape, generator=self.g, device="cuda") * (high - low) + low


def _starts(lengths):
    return torch.tensor([0] + lengths).cumsum(0).to(torch.int32).cuda()


def prepare(case, seed):
    d = _Draws(seed)
    dt = _dtype(case)
    s = {"case": case}
    if case["op"] == "conv":
        lengths = _lengths(case, seed)
        ch, w = case["channels"], case["width"]
        s["x"] = d.normal(sum(lengths), ch, dtype=dt)
        s["weight"] = d.normal(ch, w) / math.sqrt(w)
        s["bias"] = 0.1 * d.normal(ch)
        s["history"] = d.normal(len(lengths), w - 1, ch, dtype=dt)
        s["history_out"] = torch.empty_like(s["history"])
        # sequences of one length are a batch, others are packed
        s["batch"] = (len(lengths), lengths[0]) if len(set(lengths)) == 1 else None
        s["starts"] = _starts(lengths)
    elif case["op"] in ("scan", "step"):
        h, g, n, p = case["heads"], case["groups"], case["n"], case["p"]
        lengths = _lengths(case, seed) if case["op"] == "scan" else [1] * case["seqs"]
        t = sum(lengths)
        # x, B and C are column ranges of one array, as the convolution leaves them
        rows = d.normal(t, h * p + 2 * g * n, dtype=dt)
        s["x"] = rows[:, : h * p].view(t, h, p)
        s["b"] = rows[:, h * p: h * p + g * n].view(t, g, n)
        s["c"] = rows[:, h * p + g * n:].view(t, g, n)
        s["dt"] = d.normal(t, h)
        s["a_log"] = d.uniform(1.0, 16.0, h).log()
        s["dt_bias"] = d.uniform(-6.9, -2.3, h)
        s["d_skip"] = 1.0 + 0.1 * d.normal(h)
        if case["op"] == "step":
            s["state"] = 0.5 * d.normal(t, h, n, p)
        else:
            s["init"] = 0.5 * d.normal(len(lengths), h, n, p) if case["init"] else None
            s["final"] = torch.empty(len(lengths), h, n, p, device="cuda")
            s["longest"] = max(lengths)
            s["packed"] = len(lengths) > 1
            s["starts"] = _starts(lengths)
    else:
        rows, width = case["rows"], case["width"]
        s["x"] = d.normal(rows, width, dtype=dt)
        # rows of a residual stream differ in size
        s["residual"] = (d.normal(rows, width) * d.uniform(-2.0, 3.0, rows, 1).exp()).to(dt) if case["residual"] else None
        s["weight"] = 1.0 + 0.1 * d.normal(width)
    return s


# ---------------------------------------------------------------------------
# plain forms


def _silu(x):
    return x / (1 + torch.exp(-x))


def _plain_conv(s):
    case, x, starts = s["case"], s["x"], s["starts"].long()
    w = case["width"]
    t, n = x.shape[0], starts.numel() - 1
    # every sequence's history rows, then its rows, one sequence after the other
    seq = torch.searchsorted(starts[1:].contiguous(), torch.arange(t, device=x.device), right=True)
    at = torch.arange(t, device=x.device) + (w - 1) * (seq + 1)
    lead = starts[:-1] + (w - 1) * torch.arange(n, device=x.device)
    rows = torch.empty(t + n * (w - 1), x.shape[1], device=x.device, dtype=x.dtype)
    tail = torch.arange(w - 1, device=x.device)
    rows[(lead[:, None] + tail).reshape(-1)] = s["history"].reshape(n * (w - 1), -1)
    rows[at] = x
    y = (rows.unfold(0, w, 1)[at - (w - 1)].float() * s["weight"]).sum(-1) + s["bias"]
    if case["silu"]:
        y = _silu(y)
    ends = starts[1:] + (w - 1) * torch.arange(n, device=x.device)
    return y.to(x.dtype), rows[ends[:, None] + tail]


def _plain_dt(s):
    return torch.logaddexp(s["dt"].double() + s["dt_bias"].double(), torch.zeros((), device="cuda", dtype=torch.float64))


def _plain_scan(s):
    case, starts = s["case"], s["starts"].long()
    h, g, n, p = case["heads"], case["groups"], case["n"], case["p"]
    t, k, dev = s["x"].shape[0], starts.numel() - 1, s["x"].device
    nc = max(1, -(-s["longest"] // CHUNK))
    # tokens laid out as [sequence, block, place], what is behind a sequence's end as zeros
    place = torch.arange(nc * CHUNK, device=dev)
    src = (starts[:-1, None] + place).clamp(max=t - 1)
    live = place < (starts[1:] - starts[:-1])[:, None]

    def blocks(v, heads):
        v = v[src] * live.view(k, -1, *[1] * (v.dim() - 1))
        v = v.view(k, nc, CHUNK, heads, -1).permute(0, 1, 3, 2, 4)
        return v

    x = blocks(s["x"].float(), h)
    b = blocks(s["b"].float(), g).repeat_interleave(h // g, 2)
    c = blocks(s["c"].float(), g).repeat_interleave(h // g, 2)
    dt = blocks(_plain_dt(s), h).squeeze(-1)  # [k, nc, h, CHUNK]
    cum = (-torch.exp(s["a_log"].double())[:, None] * dt).cumsum(-1)
    causal = torch.ones(CHUNK, CHUNK, device=dev, dtype=torch.bool).tril()
    decay = torch.where(causal, cum[..., :, None] - cum[..., None, :], -math.inf).exp()
    mix = torch.matmul(c, b.transpose(-1, -2)) * (decay * dt[..., None, :]).float()
    y = torch.matmul(mix, x)
    last = cum[..., -1]
    ends = torch.matmul(b.transpose(-1, -2), x * ((last[..., None] - cum).exp() * dt).float()[..., None])
    # the state before block i: all earlier blocks' ends and the first state, each decayed up to there
    total = torch.cat([torch.zeros_like(last[:, :1]), last.cumsum(1)], 1).permute(0, 2, 1)  # [k, h, nc + 1]
    before = torch.ones(nc + 1, nc, device=dev, dtype=torch.bool).tril(-1)
    carry = torch.where(before, total[..., :, None] - total[..., None, 1:], -math.inf).exp().float()
    states = torch.matmul(carry, ends.permute(0, 2, 1, 3, 4).reshape(k, h, nc, n * p)).view(k, h, nc + 1, n, p)
    if s["init"] is not None:
        states = states + total.exp().float()[..., None, None] * s["init"][:, :, None]
    y = y + torch.matmul(c, states[:, :, :-1].transpose(1, 2)) * cum.exp().float()[..., None]
    y = y + s["d_skip"][:, None, None] * x
    seq = torch.searchsorted(starts[1:].contiguous(), torch.arange(t, device=dev), right=True)
    at = torch.arange(t, device=dev) - starts[seq] + seq * nc * CHUNK
    y = y.permute(0, 1, 3, 2, 4).reshape(k * nc * CHUNK, h, p)[at]
    return y.to(s["x"].dtype), states[:, :, -1].contiguous()


def _plain_step(s):
    case = s["case"]
    rep = case["heads"] // case["groups"]
    x, dt = s["x"].float(), _plain_dt(s)
    b, c = (s[v].float().repeat_interleave(rep, 1) for v in ("b", "c"))
    decay = torch.exp(-torch.exp(s["a_log"].double()) * dt).float()
    state = decay[..., None, None] * s["state"] + (dt.float()[..., None] * b)[..., None] * x[..., None, :]
    s["state"].copy_(state)
    y = (state * c[..., None]).sum(2) + s["d_skip"][:, None] * x
    return y.to(s["x"].dtype), s["state"]


def _plain_norm(s):
    case, x = s["case"], s["x"]
    r = x.float() + s["residual"].float() if case["residual"] else x.float()
    y = r / torch.sqrt(r.square().mean(-1, keepdim=True) + 1e-6) * s["weight"]
    got = {}
    if case["residual"]:
        got["residual"] = r.to(x.dtype)
    if case["out"]:
        got["out"] = y.to(x.dtype)
    if case["scales"] == "row":
        got["scales"] = y.abs().amax(-1).clamp(min=SCALE_FLOOR) / E4M3_MAX
        got["quant"] = (y / got["scales"][:, None]).to(torch.float8_e4m3fn)
    elif case["scales"] == "group":
        rows, width = y.shape
        part = torch.cat([y, y.new_zeros(rows, -width % GROUP)], 1).view(rows, -1, GROUP)
        got["scales"] = part.abs().amax(-1).clamp(min=SCALE_FLOOR) / E4M3_MAX
        got["quant"] = (part / got["scales"][..., None]).view(rows, -1)[:, :width].contiguous().to(torch.float8_e4m3fn)
    return got


# ---------------------------------------------------------------------------
# the library's calls


def _own_conv(s):
    import gated_deltanet_02_amd as G

    case, x = s["case"], s["x"]
    if s["batch"]:
        y = G.gdn_short_conv(x.view(*s["batch"], -1), s["weight"], s["bias"], state_in=s["history"], state_out=s["history_out"], silu=case["silu"]).view(x.shape)
    else:
        y = G.gdn_short_conv(x, s["weight"], s["bias"], cu_seqlens=s["starts"], state_in=s["history"], state_out=s["history_out"], silu=case["silu"])
    return y, s["history_out"]


def _own_scan(s):
    import gated_deltanet_02_amd as G

    return G.gdn_ssm_prefill(s["x"], s["dt"], s["b"], s["c"], s["a_log"], dt_bias=s["dt_bias"], d_skip=s["d_skip"], cu_seqlens=s["starts"] if s["packed"] else None, init_state=s["init"], final_state=s["final"])


def _own_step(s):
    import gated_deltanet_02_amd as G

    y = G.gdn_ssm_decode(s["x"], s["dt"], s["b"], s["c"], s["state"], s["a_log"], dt_bias=s["dt_bias"], d_skip=s["d_skip"])
    return y, s["state"]


def _own_norm(s):
    import gated_deltanet_02_amd as G

    case, x = s["case"], s["x"]
    rows, width = x.shape
    got = {}
    if case["residual"]:
        got["residual"] = torch.empty_like(x)
    if case["out"]:
        got["out"] = torch.empty_like(x)
    if case["scales"] != "none":
        got["quant"] = torch.empty(rows, width, dtype=torch.float8_e4m3fn, device=x.device)
        got["scales"] = torch.empty((rows,) if case["scales"] == "row" else (rows, -(-width // GROUP)), device=x.device)
    G.gdn_add_rms_norm(x, s["residual"], s["weight"], residual_out=got.get("residual"), out=got.get("out"), out_q=got.get("quant"), scales=got.get("scales"))
    return got


def run(state):
    if own:
        return {"conv": _own_conv, "scan": _own_scan, "step": _own_step, "norm": _own_norm}[state["case"]["op"]](state)
    return {"conv": _plain_conv, "scan": _plain_scan, "step": _plain_step, "norm": _plain_norm}[state["case"]["op"]](state)


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "conv":
        lengths = _lengths(case, 0)
        t, ch, w = sum(lengths), case["channels"], case["width"]
        return {"bytes": 2 * t * ch * size + 2 * len(lengths) * (w - 1) * ch * size + ch * (w + 1) * 4, "flops": 2 * t * ch * w}
    if case["op"] in ("scan", "step"):
        h, g, n, p = case["heads"], case["groups"], case["n"], case["p"]
        lengths = _lengths(case, 0) if case["op"] == "scan" else [1] * case["seqs"]
        t = sum(lengths)
        states = len(lengths) * h * n * p * 4
        moved = 2 * states if case["op"] == "step" or case["init"] else states
        return {"bytes": 2 * t * h * p * size + 2 * t * g * n * size + 4 * t * h + 12 * h + moved, "flops": t * h * (4 * n * p + 2 * p)}
    rows, width = case["rows"], case["width"]
    moved = rows * width * (size * (1 + 2 * case["residual"] + case["out"]) + (case["scales"] != "none")) + 4 * width
    moved += 4 * rows * (0 if case["scales"] == "none" else 1 if case["scales"] == "row" else -(-width // GROUP))
    return {"bytes": moved, "flops": 6 * rows * width}


# ---------------------------------------------------------------------------
# 64 bits, from the definitions


def exact(case, seed):
    s = prepare(case, seed)
    d = lambda v: None if v is None else v.double()  # noqa: E731
    if case["op"] == "conv":
        lengths = _lengths(case, seed)
        w, t0, ys, tails = case["width"], 0, [], []
        taps, bias = d(s["weight"]), d(s["bias"])
        for i, length in enumerate(lengths):
            e = torch.cat([s["history"][i], s["x"][t0: t0 + length]])
            y = bias.expand(length, -1).clone()
            for j in range(w):
                y += taps[:, j] * e[j: j + length].double()
            # returned in 32 bits, a sixteenth of a 16-bit step and less
            ys.append((y * torch.sigmoid(y) if case["silu"] else y).to(torch.float64 if case["dtype"] == "f32" else torch.float32))
            tails.append(e[length:])
            t0 += length
        return torch.cat(ys), torch.stack(tails).double()
    if case["op"] in ("scan", "step"):
        lengths = _lengths(case, seed) if case["op"] == "scan" else [1] * case["seqs"]
        h, rep = case["heads"], case["heads"] // case["groups"]
        starts = torch.tensor([0] + lengths).cumsum(0).tolist()
        dt = torch.nn.functional.softplus(d(s["dt"]) + d(s["dt_bias"]), threshold=50)
        decay = torch.exp(-torch.exp(d(s["a_log"])) * dt)
        state = d(s["state"]) if case["op"] == "step" else d(s["init"]) if case["init"] else torch.zeros(len(lengths), h, case["n"], case["p"], device="cuda", dtype=torch.float64)
        # the longest sequences first, so that those with a token left are a leading range
        order = sorted(range(len(lengths)), key=lambda i: -lengths[i])
        state = state[order]
        first = torch.tensor([starts[i] for i in order]).cuda()
        y = torch.empty(s["x"].shape, device="cuda", dtype=torch.float64)
        live = len(order)
        for t in range(max(lengths)):
            while lengths[order[live - 1]] <= t:
                live -= 1
            at = first[:live] + t
            x, b, c = (d(s[v][at]) for v in ("x", "b", "c"))
            if rep > 1:
                b, c = b.repeat_interleave(rep, 1), c.repeat_interleave(rep, 1)
            now = state[:live]
            now.mul_(decay[at][..., None, None])
            now.addcmul_((dt[at][..., None] * b)[..., None], x[..., None, :])
            y[at] = torch.matmul(c[..., None, :], now)[..., 0, :] + d(s["d_skip"])[:, None] * x
        back = torch.empty_like(state)
        back[torch.tensor(order).cuda()] = state
        return y, back
    r = d(s["x"]) + (d(s["residual"]) if case["residual"] else 0)
    y = r * torch.rsqrt(torch.mean(r * r, 1, keepdim=True) + 1e-6) * d(s["weight"])
    got = {}
    if case["residual"]:
        got["residual"] = r
    if case["out"]:
        got["out"] = y
    if case["scales"] != "none":
        cuts = [y] if case["scales"] == "row" else list(torch.split(y, GROUP, 1))
        scales = [v.abs().amax(1).clamp(min=SCALE_FLOOR) / E4M3_MAX for v in cuts]
        got["scales"] = scales[0] if case["scales"] == "row" else torch.stack(scales, 1)
        got["quant"] = torch.cat([v / f[:, None] for v, f in zip(cuts, scales)], 1)
    return got
