"""float64 references of the attention over a paged cache and of the cache's
bookkeeping, in numpy and plain Python."""
from __future__ import annotations

import numpy as np


def seen(place: int, n: int, window: int = 0, sinks: int = 0) -> np.ndarray:
    """The keys 0 .. n - 1 that the query at ``place`` sees."""
    j = np.arange(n)
    s = j <= place
    if window > 0:
        s &= (j > place - window) | (j < sinks)
    return s


def attention(q, k, v, first: int, window: int = 0, sinks: int = 0, scale=None):
    """q [rows, H, d] at the places first, first + 1, ... against k, v [n, Hk,
    d].  Returns (out, M, S): M the sum of the weights times |v|, S the largest
    scale sum |q k| of a row (what errors scale with)."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    rows, H, d = q.shape
    n, Hk = k.shape[:2]
    scale = d ** -0.5 if scale is None else scale
    out, M, S = np.zeros((rows, H, d)), np.zeros((rows, H, d)), np.zeros((rows, H, 1))
    see = np.stack([seen(first + r, n, window, sinks) for r in range(rows)]) if rows else np.zeros((0, n), bool)
    any_seen = see.any(1)
    if n == 0:
        return out, M, S
    for h in range(H):
        kh, vh = k[:, h // (H // Hk)], v[:, h // (H // Hk)]
        s = np.where(see, scale * (q[:, h] @ kh.T), -np.inf)
        top = np.where(any_seen, s.max(1), 0.0)
        w = np.exp(s - top[:, None])
        total = np.where(any_seen, w.sum(1), 1.0)
        w /= total[:, None]
        out[:, h] = w @ vh
        M[:, h] = w @ np.abs(vh)
        S[:, h, 0] = (np.abs(scale) * (np.abs(q[:, h]) @ np.abs(kh).T) * see).max(1)
    return out, M, S


def gather(cache, row, n: int):
    """The first n rows of a sequence in a cache [pages, S, Hk, d]."""
    size = cache.shape[1]
    return np.stack([cache[row[p // size], p % size] for p in range(n)]) if n else cache[:0].reshape(0, *cache.shape[2:])


def plan(ctx, starts, table, free, n_free: int, page: int, t: int):
    """Serial reference of the plan; ``starts`` [N + 1].  Returns (table, lens,
    slots, left)."""
    table, stack = table.copy(), list(free[:n_free])
    lens, slots = [], np.full(t, -1, np.int64)
    blocked = False
    for i, c in enumerate(ctx):
        new = starts[i + 1] - starts[i]
        have, need = -(-c // page), -(-(c + new) // page)
        want = need - have
        if need > table.shape[1]:
            lens.append(c)
            continue
        if want > 0 and (blocked or want > len(stack)):
            blocked = True
            lens.append(c)
            continue
        for j in range(have, need):
            table[i, j] = stack.pop()
        for x in range(new):
            p = c + x
            if table[i, p // page] >= 0:
                slots[starts[i] + x] = int(table[i, p // page]) * page + p % page
        lens.append(c + new)
    return table, np.array(lens, np.int32), slots, len(stack)


def release(done, lens, table, free, n_free: int, page: int):
    """Serial reference of the release; returns (lens, table, free, n_free)."""
    lens, table, free = lens.copy(), table.copy(), free.copy()
    for i, f in enumerate(done):
        if not f:
            continue
        for j in range(min(-(-int(lens[i]) // page), table.shape[1])):
            if table[i, j] >= 0 and n_free < len(free):
                free[n_free] = table[i, j]
                n_free += 1
            table[i, j] = -1
        lens[i] = 0
    return lens, table, free, n_free
