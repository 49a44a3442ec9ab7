"""The attention layers that a hybrid model has between its recurrent ones, as measured cases: block tables and slot maps made from request lengths, the store of new keys and values into a
paged cache, attention of one new token over that cache, and causal attention of prompts with a sliding window and first tokens that stay visible, over the prompts alone or behind what the cache
holds. Each is computed either in its plain form (elementary torch operations in float32) or by the library's entry points."""
import math

import torch

own = False


def _spread(count, low, high, seed):
    """Lengths spread evenly over [low, high] in an order that the seed shuffles: their total does not depend on the seed."""
    lengths = torch.linspace(low, high, count).round().to(torch.int64)
    return lengths[torch.randperm(count, generator=torch.Generator().manual_seed(seed))].tolist()


def _lengths(text, seed):
    """Lengths written out ("1,63,64"), or "spread COUNT LOW HIGH"."""
    if text.startswith("spread"):
        count, low, high = (int(v) for v in text.split()[1:])
        return _spread(count, low, high, seed)
    return [int(v) for v in text.split(",")]


def _requests(case, seed):
    """Each request's tokens in the cache and its new ones."""
    new = _lengths(case["new"], seed + 1)
    past = _lengths(case["past"], seed) if case["past"] else [0] * len(new)
    return past, new


def listed():
    plan = {"op": "plan", "short": False}
    store = {"op": "store", "dtype": "bf16"}
    attend = {"op": "attend", "dtype": "bf16", "window": 0, "sinks": 0}
    prompt = {"op": "prompt", "dtype": "bf16", "window": 0, "sinks": 0, "past": "", "page": 0}
    return [
        # one new token for each of 256 running sequences
        {"name": "plan step", **plan, "past": "spread 256 200 4096", "new": ",".join(["1"] * 256), "page": 16},
        # a packed batch of new prompts
        {"name": "plan prompts", **plan, "past": "", "new": "spread 64 200 4096", "page": 64},
        # the new token's keys and values of 256 running sequences
        {"name": "store step", **store, "past": "spread 256 200 4096", "new": ",".join(["1"] * 256), "kv": 8, "d": 128, "page": 16},
        # those of a packed batch of new prompts
        {"name": "store prompts", **store, "past": "", "new": "spread 64 200 4096", "kv": 8, "d": 128, "page": 64},
        # a single running sequence: its latency
        {"name": "attend one", **attend, "past": "4096", "heads": 32, "kv": 8, "d": 128, "page": 64},
        # a serving batch of ragged lengths, small pages
        {"name": "attend batch", **attend, "past": "spread 256 200 4096", "heads": 32, "kv": 8, "d": 128, "page": 16},
        # a few long contexts beside a short one, large heads
        {"name": "attend long", **attend, "past": "131072,100001,65537,1000", "heads": 16, "kv": 2, "d": 256, "page": 64},
        # a window with first tokens that stay, six heads to a key head, pages that are no power of two, float32
        {"name": "attend window", **attend, "dtype": "f32", "past": "spread 64 1000 32768", "heads": 48, "kv": 8, "d": 64, "page": 48, "window": 1024, "sinks": 4},
        # one prompt at the default length limit
        {"name": "prompt", **prompt, "new": "4096", "heads": 16, "kv": 4, "d": 128},
        # the longest prompt, with a window and first tokens that stay
        {"name": "prompt window", **prompt, "new": "16384", "heads": 16, "kv": 16, "d": 128, "window": 1024, "sinks": 4},
        # prompts in chunks behind what the cache holds of them, large heads, small pages
        {"name": "prompt chunks", **prompt, "past": "spread 16 0 6144", "new": "spread 16 200 2048", "heads": 16, "kv": 2, "d": 256, "page": 16},
        # ragged lengths around the tile size, a window that ends inside tiles, float32
        {"name": "prompt edge", **prompt, "dtype": "f32", "new": "1,63,64,65,1000", "heads": 8, "kv": 8, "d": 64, "window": 100, "sinks": 2},
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["plan", "store", "attend", "attend", "prompt", "prompt"])
    page = rng.choice([8, 16, 16, 32, 48, 64, 128])
    if op in ("plan", "store"):
        if rng.random() < 0.5:
            # running sequences, one new token each
            seqs = _log_int(rng, 1, 256)
            past, new = "spread %d %d %d" % (seqs, rng.randint(0, 200), rng.randint(201, 4096)), ",".join(["1"] * seqs)
        else:
            # a few requests with new tokens behind their cached ones, some without any
            seqs = rng.randint(1, 32)
            lengths = [_log_int(rng, 1, 4096) if rng.random() < 0.9 else 0 for _ in range(seqs)]
            lengths[rng.randrange(seqs)] = _log_int(rng, 1, 4096)
            past, new = ",".join(str(rng.randint(0, 2048)) for _ in range(seqs)), ",".join(str(v) for v in lengths)
        case = {"op": op, "past": past, "new": new, "page": page}
        if op == "plan":
            return {**case, "short": rng.random() < 0.3}
        return {**case, "dtype": rng.choice(["bf16", "bf16", "f32"]), "kv": rng.choice([1, 2, 4, 8]), "d": rng.choice([64, 128, 256])}
    dtype, d, kv = rng.choice(["bf16", "bf16", "f32"]), rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 6, 8])
    window, sinks = (_log_int(rng, 16, 4096), rng.choice([0, 1, 4, 64])) if rng.random() < 0.5 else (0, 0)
    case = {"op": op, "dtype": dtype, "heads": kv * group, "kv": kv, "d": d, "window": window, "sinks": sinks}
    if op == "attend":
        # what the cache holds: at most 1 GB of keys and values
        tokens = (1 << 30) // (2 * kv * d * (2 if dtype == "bf16" else 4))
        kind = rng.random()
        if kind < 0.3:
            past = str(_log_int(rng, 1, min(131072, tokens)))
        elif kind < 0.65:
            past = ",".join(str(_log_int(rng, 1, min(32768, tokens // 8))) for _ in range(rng.randint(2, 8)))
        else:
            seqs = _log_int(rng, 9, 256)
            past = "spread %d %d %d" % (seqs, rng.randint(1, 200), min(rng.randint(201, 8192), max(201, 2 * tokens // seqs - 201)))
        return {**case, "past": past, "page": page}
    # prompts: at most 2^30 pairs of a query and a key over all heads
    most = (1 << 30) // case["heads"]
    kind = rng.random()
    if kind < 0.35:
        past, new = "", str(_log_int(rng, 1, min(8192, int(math.sqrt(most)))))
    else:
        seqs = rng.randint(2, 16)
        top = min(4096, int(math.sqrt(most / seqs)))
        new = ",".join(str(_log_int(rng, 1, top) if rng.random() < 0.9 else 0) for _ in range(seqs - 1)) + "," + str(rng.randint(1, top))
        past = ",".join(str(rng.randint(0, top)) for _ in range(seqs)) if kind > 0.65 else ""
    return {**case, "past": past, "new": new, "page": page if past else 0}


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


class _Draws:
    """Seeded draws on the GPU."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(self, *shape, dtype=torch.float32):
        return torch.randn(*shape, generator=self.g, device="cuda", dtype=dtype)

    def order(self, n):
        return torch.randperm(n, generator=self.g, device="cuda")


def _starts(lengths):
    return torch.tensor([0] + lengths).cumsum(0).to(torch.int32).cuda()


def _ceil(a, b):
    return -(-a // b)


def _pool(d, tokens, page, spare):
    """A pool of pages in no order, of which the requests hold those for their tokens: the table of each request's pages (what it does not hold is -1), the pages that nobody holds, and the
    number of pages."""
    have = [_ceil(t, page) for t in tokens]
    pages = sum(have) + spare
    order = d.order(pages).to(torch.int32)
    width = max(1, max(have))
    col = torch.arange(width)
    held = (col < torch.tensor(have)[:, None]).cuda()
    table = torch.full((len(tokens), width), -1, dtype=torch.int32, device="cuda")
    table[held] = order[: sum(have)]
    return table, order[sum(have):].contiguous(), pages


def prepare(case, seed):
    d = _Draws(seed)
    s = {"case": case}
    op = case["op"]
    if op == "attend":
        past = _lengths(case["past"], seed)
        dt = _dtype(case)
        s["table"], _, pages = _pool(d, past, case["page"], 1)
        s["lens"] = torch.tensor(past, dtype=torch.int32).cuda()
        s["k"], s["v"] = (d.normal(pages, case["page"], case["kv"], case["d"], dtype=dt) for _ in range(2))
        # the queries are a column range of the projection's output
        s["q"] = d.normal(len(past), (case["heads"] + 2 * case["kv"]) * case["d"], dtype=dt)[:, : case["heads"] * case["d"]].view(len(past), case["heads"], case["d"])
        return s
    past, new = _requests(case, seed)
    t, n = sum(new), len(new)
    s["starts"] = _starts(new)
    if op == "plan":
        ahead = [_ceil(a + b, case["page"]) for a, b in zip(past, new)]
        wanted = sum(ahead) - sum(_ceil(a, case["page"]) for a in past)
        held, s["free"], _ = _pool(d, past, case["page"], max(1, wanted // 2 if case["short"] else wanted + 7))
        s["table"] = torch.full((n, max(1, max(ahead))), -1, dtype=torch.int32, device="cuda")
        s["table"][:, : held.shape[1]] = held[:, : s["table"].shape[1]]
        s["n_free"] = torch.tensor([s["free"].numel()], dtype=torch.int32).cuda()
        s["past"] = torch.tensor(past, dtype=torch.int32).cuda()
        s["t"], s["step"] = t, all(v == 1 for v in new)
        return s
    dt = _dtype(case)
    if op == "store":
        table, _, pages = _pool(d, [a + b for a, b in zip(past, new)], case["page"], 1)
        seq = torch.repeat_interleave(torch.arange(n), torch.tensor(new))
        at = torch.arange(t) - s["starts"].cpu().long()[seq] + torch.tensor(past)[seq]
        seq, at = seq.cuda(), at.cuda()
        s["slots"] = table[seq, at // case["page"]].long() * case["page"] + at % case["page"]
        # a request that got no pages: its rows are not stored
        if n > 2:
            s["slots"][seq == n // 2] = -1
        rows = d.normal(t, 4 * case["kv"] * case["d"], dtype=dt)
        s["k"], s["v"] = (rows[:, i * case["kv"] * case["d"]: (i + 1) * case["kv"] * case["d"]].view(t, case["kv"], case["d"]) for i in (2, 3))
        s["k_cache"], s["v_cache"] = (d.normal(pages, case["page"], case["kv"], case["d"], dtype=dt) for _ in range(2))
        return s
    rows = d.normal(t, (case["heads"] + 2 * case["kv"]) * case["d"], dtype=dt)
    cut = lambda a, b: rows[:, a * case["d"]: b * case["d"]].view(t, b - a, case["d"])  # noqa: E731
    s["q"], s["k"], s["v"] = cut(0, case["heads"]), cut(case["heads"], case["heads"] + case["kv"]), cut(case["heads"] + case["kv"], case["heads"] + 2 * case["kv"])
    s["longest"], s["packed"] = max(new), n > 1
    s["most"] = max(a + b for a, b in zip(past, new))
    s["lens"] = torch.tensor([a + b for a, b in zip(past, new)], dtype=torch.int32).cuda()
    s["table"] = None
    if case["page"]:
        # the cache holds the earlier tokens and, stored before this call, the new ones
        s["table"], _, pages = _pool(d, [a + b for a, b in zip(past, new)], case["page"], 1)
        s["k"], s["v"] = (d.normal(pages, case["page"], case["kv"], case["d"], dtype=dt) for _ in range(2))
    return s


# ---------------------------------------------------------------------------
# plain forms


def _plain_plan(s):
    page, table = s["case"]["page"], s["table"]
    starts, past = s["starts"].long(), s["past"].long()
    new = starts[1:] - starts[:-1]
    have, need = (past + page - 1) // page, (past + new + page - 1) // page
    fits = need <= table.shape[1]
    extra = torch.where(fits, need - have, 0)
    upto = extra.cumsum(0)
    # a request gets all of its pages or none, in the order of the requests
    served = fits & ((extra == 0) | (upto <= s["n_free"]))
    taken = torch.where(served, upto * (extra > 0), 0).amax()
    lens = torch.where(served, past + new, past)
    t = s["t"]
    seq = torch.searchsorted(starts[1:].contiguous(), torch.arange(t, device=table.device), right=True)
    at = past[seq] + torch.arange(t, device=table.device) - starts[seq]
    col = at // page
    fresh = col >= have[seq]
    pick = s["n_free"] - 1 - (upto - extra)[seq] - (col - have[seq])
    got = s["free"].long()[pick.clamp(min=0, max=s["free"].numel() - 1)]
    old = table[seq, col.clamp(max=table.shape[1] - 1)].long()
    entry = torch.where(fresh, got, old)
    ok = served[seq]
    slots = torch.where(ok, entry * page + at % page, -1)
    # every fresh page's first token writes its entry, the others write what is there
    first = ok & fresh & (at % page == 0)
    table.view(-1)[(seq * table.shape[1] + col)[first]] = got[first].to(torch.int32)
    return table, lens.to(torch.int32), slots, (s["n_free"] - taken).to(torch.int32)


def _plain_store(s):
    ok = s["slots"] >= 0
    at = s["slots"][ok]
    for cache, rows in ((s["k_cache"], s["k"]), (s["v_cache"], s["v"])):
        cache.view(-1, *cache.shape[2:])[at] = rows[ok]
    return s["k_cache"], s["v_cache"]


def _softmax(scores, seen):
    """Weights of the seen columns in place; rows that see nothing are zeros."""
    scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    scores.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    return scores.div_(scores.sum(-1, keepdim=True).clamp(min=1e-30))


def _seen(col, at, case):
    """Whether the token at place `at` sees the one at `col`."""
    seen = col <= at
    if case["window"]:
        seen = seen & ((col > at - case["window"]) | (col < case["sinks"]))
    return seen


def _gathered(s, cache, most):
    """A cache's rows as [sequence, head, place, d]; what is behind a sequence's end as zeros."""
    n, page = s["lens"].numel(), s["case"]["page"]
    col = torch.arange(_ceil(most, page), device="cuda")
    rows = cache[s["table"][:, : col.numel()].clamp(min=0).long()].view(n, -1, *cache.shape[2:])
    live = torch.arange(rows.shape[1], device="cuda") < s["lens"][:, None]
    return torch.where(live[..., None, None], rows, 0).float().permute(0, 2, 1, 3)


def _plain_attend(s):
    case, q = s["case"], s["q"].float()
    n, h, d = q.shape
    most = s["table"].shape[1] * case["page"]
    k, v = _gathered(s, s["k"], most), _gathered(s, s["v"], most)
    scores = torch.matmul(q.view(n, case["kv"], -1, d) / math.sqrt(d), k.transpose(-1, -2))
    at = s["lens"][:, None, None, None] - 1
    w = _softmax(scores, _seen(torch.arange(k.shape[2], device="cuda"), at, case))
    return torch.matmul(w, v).reshape(n, h, d).to(s["q"].dtype)


def _plain_prompt(s):
    case, q, starts = s["case"], s["q"], s["starts"].long()
    t, h, d = q.shape
    n, g, kv = starts.numel() - 1, case["heads"] // case["kv"], case["kv"]
    lens, new = s["lens"].long(), starts[1:] - starts[:-1]
    row = torch.arange(s["longest"], device="cuda")
    src = (starts[:-1, None] + row).clamp(max=t - 1)
    at = (lens - new)[:, None] + row  # the rows' places in their sequences
    if case["page"]:
        k, v = _gathered(s, s["k"], s["most"]), _gathered(s, s["v"], s["most"])
    else:
        live = (row < new[:, None])[..., None, None]
        k, v = (torch.where(live, s[x][src], 0).float().permute(0, 2, 1, 3) for x in ("k", "v"))
    qs = (q[src].float() / math.sqrt(d)).view(n, -1, kv, g, d).permute(0, 2, 3, 1, 4)  # [n, kv, g, row, d]
    scores = torch.matmul(qs, k[:, :, None].transpose(-1, -2))
    w = _softmax(scores, _seen(torch.arange(k.shape[2], device="cuda"), at[:, None, None, :, None], case))
    y = torch.matmul(w, v[:, :, None]).permute(0, 3, 1, 2, 4).reshape(n * s["longest"], h, d)
    seq = torch.searchsorted(starts[1:].contiguous(), torch.arange(t, device="cuda"), right=True)
    return y[seq * s["longest"] + torch.arange(t, device="cuda") - starts[seq]].to(q.dtype)


# ---------------------------------------------------------------------------
# the library's calls


def _own_plan(s):
    import gated_deltanet_02_amd as G

    lens, slots, left = G.gdn_cache_plan(s["past"], s["case"]["page"], s["table"], s["free"], s["n_free"], cu_seqlens=None if s["step"] else s["starts"], n_tokens=s["t"])
    return s["table"], lens, slots, left


def _own_store(s):
    import gated_deltanet_02_amd as G

    G.gdn_cache_store(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"])
    return s["k_cache"], s["v_cache"]


def _own_attend(s):
    import gated_deltanet_02_amd as G

    case = s["case"]
    return G.gdn_attn_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], window=case["window"], sinks=case["sinks"])


def _own_prompt(s):
    import gated_deltanet_02_amd as G

    case = s["case"]
    cache = {"block_table": s["table"], "seq_lens": s["lens"]} if case["page"] else {}
    return G.gdn_attn_prefill(s["q"], s["k"], s["v"], cu_seqlens=s["starts"] if s["packed"] or cache else None, window=case["window"], sinks=case["sinks"], **cache)


def run(state):
    if own:
        return {"plan": _own_plan, "store": _own_store, "attend": _own_attend, "prompt": _own_prompt}[state["case"]["op"]](state)
    return {"plan": _plain_plan, "store": _plain_store, "attend": _plain_attend, "prompt": _plain_prompt}[state["case"]["op"]](state)


def _sights(past, new, window, sinks):
    """How many tokens the new ones of a sequence see, together."""
    if new == 0:
        return 0
    at = torch.arange(past, past + new, dtype=torch.int64) + 1
    if window:
        at = torch.minimum(at, window + (at - window).clamp(min=0, max=sinks))
    return int(at.sum())


def work(case):
    if case["op"] == "attend":
        past = _lengths(case["past"], 0)
        size = 2 if case["dtype"] == "bf16" else 4
        seen = sum(_sights(p - 1, 1, case["window"], case["sinks"]) for p in past)
        moved = 2 * seen * case["kv"] * case["d"] * size + 2 * len(past) * case["heads"] * case["d"] * size
        return {"bytes": moved + 4 * _ceil(seen, case["page"]) + 4 * len(past), "flops": 4 * seen * case["heads"] * case["d"]}
    past, new = _requests(case, 0)
    t, n = sum(new), len(new)
    if case["op"] == "plan":
        fresh = sum(_ceil(a + b, case["page"]) - _ceil(a, case["page"]) for a, b in zip(past, new))
        # lengths and starts read, lengths and a slot a token written; a page a fresh entry moved, an entry read for a token in a page held before
        return {"bytes": 12 * n + 8 * t + 8 * fresh + 4 * n, "flops": 4 * t + 8 * n}
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "store":
        return {"bytes": 4 * t * case["kv"] * case["d"] * size + 8 * t, "flops": t}
    keys = sum(a + b for a, b in zip(past, new)) if not case["window"] else sum(min(a + b, b + case["window"] + case["sinks"]) for a, b in zip(past, new) if b)
    seen = sum(_sights(a, b, case["window"], case["sinks"]) for a, b in zip(past, new))
    return {"bytes": 2 * t * case["heads"] * case["d"] * size + 2 * keys * case["kv"] * case["d"] * size, "flops": 4 * seen * case["heads"] * case["d"]}


# ---------------------------------------------------------------------------
# 64 bits, from the definitions


def _rows_of(s, cache, i, length):
    """The first `length` rows of sequence i in a cache."""
    places = torch.arange(length, device="cuda")
    return cache[s["table"][i].long()[places // s["case"]["page"]], places % s["case"]["page"]].double()


def _attention(q, k, v, first, window, sinks):
    """Rows [rows, heads, d] at the places first, first + 1, ... against keys and values [places, kv, d]."""
    rows, heads, d = q.shape
    rep = heads // k.shape[1]
    out = torch.empty_like(q)
    place = torch.arange(first, first + rows, device="cuda")[:, None]
    key = torch.arange(k.shape[0], device="cuda")[None, :]
    hidden = key > place
    if window > 0:
        hidden |= (place - key >= window) & (key >= sinks)
    for h in range(heads):
        logits = q[:, h] @ k[:, h // rep].T * d ** -0.5
        out[:, h] = torch.softmax(logits.masked_fill(hidden, -math.inf), 1) @ v[:, h // rep]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        past = _lengths(case["past"], seed)
        out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        for i, length in enumerate(past):
            k, v = _rows_of(s, s["k"], i, length), _rows_of(s, s["v"], i, length)
            if case["window"] and length > case["window"] + case["sinks"]:
                k, v = (torch.cat([x[: case["sinks"]], x[length - case["window"]:]]) for x in (k, v))
            rep = case["heads"] // case["kv"]
            logits = s["q"][i].double().view(case["kv"], rep, -1) @ k.permute(1, 2, 0) * case["d"] ** -0.5
            out[i] = (torch.softmax(logits, -1) @ v.permute(1, 0, 2)).reshape(case["heads"], -1)
        return out
    past, new = _requests(case, seed)
    if case["op"] == "plan":
        free, left = s["free"].tolist(), int(s["n_free"])
        table, lens, slots = s["table"].cpu(), [], []
        stack = free[:left]
        blocked = False
        for i, (a, b) in enumerate(zip(past, new)):
            have, need = _ceil(a, case["page"]), _ceil(a + b, case["page"])
            if need > table.shape[1] or (need > have and (blocked or need - have > len(stack))):
                blocked = blocked or need <= table.shape[1]
                lens.append(a)
                slots.append(torch.full((b,), -1))
                continue
            for j in range(have, need):
                table[i, j] = stack.pop()
            lens.append(a + b)
            at = torch.arange(a, a + b)
            slots.append(table[i].long()[at // case["page"]] * case["page"] + at % case["page"])
        return table, torch.tensor(lens, dtype=torch.int32), torch.cat(slots), torch.tensor([len(stack)], dtype=torch.int32)
    if case["op"] == "store":
        got = []
        for cache, rows in ((s["k_cache"], s["k"]), (s["v_cache"], s["v"])):
            flat = cache.flatten(0, 1)
            src = torch.full((flat.shape[0],), -1, dtype=torch.int64, device="cuda")
            src[s["slots"][s["slots"] != -1]] = (s["slots"] != -1).nonzero()[:, 0]
            got.append(torch.where((src >= 0)[:, None, None], rows[src.clamp(min=0)], flat).view(cache.shape))
        return tuple(got)
    out, t0 = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda"), 0
    for i, (a, b) in enumerate(zip(past, new)):
        if case["page"]:
            k, v = _rows_of(s, s["k"], i, a + b), _rows_of(s, s["v"], i, a + b)
        else:
            k, v = s["k"][t0: t0 + b].double(), s["v"][t0: t0 + b].double()
        out[t0: t0 + b] = _attention(s["q"][t0: t0 + b].double(), k, v, a, case["window"], case["sinks"])
        t0 += b
    return out
