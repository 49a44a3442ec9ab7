"""The float64 references of the attention and of the cache's bookkeeping
against independent forms (CPU)."""
import numpy as np
import pytest

from oracle import attention as A


def softmax_rows(q, k, v, first, window, sinks, scale):
    """Key by key in plain Python."""
    out = np.zeros(q.shape)
    H, Hk = q.shape[1], k.shape[1]
    for r in range(q.shape[0]):
        p = first + r
        for h in range(H):
            keys = [j for j in range(k.shape[0]) if j <= p and (window == 0 or p - j < window or j < sinks)]
            if not keys:
                continue
            e = [np.exp(scale * sum(q[r, h, c] * k[j, h * Hk // H, c] for c in range(q.shape[2]))) for j in keys]
            for j, w in zip(keys, e):
                out[r, h] += w / sum(e) * v[j, h * Hk // H]
    return out


@pytest.mark.parametrize("first,window,sinks", [(0, 0, 0), (3, 0, 0), (0, 2, 0), (4, 3, 1), (-2, 0, 0), (5, 1, 2)])
def test_attention_key_by_key(first, window, sinks):
    g = np.random.default_rng(1)
    n = max(0, first + 4)
    q, k, v = g.standard_normal((4, 6, 5)), g.standard_normal((n, 2, 5)), g.standard_normal((n, 2, 5))
    got, M, S = A.attention(q, k, v, first, window, sinks, 0.3)
    want = softmax_rows(q, k, v, first, window, sinks, 0.3)
    np.testing.assert_allclose(got, want, rtol=1e-12, atol=1e-12)
    assert (np.abs(got) <= M + 1e-12).all()


def test_attention_invariants():
    g = np.random.default_rng(2)
    q, k, v = g.standard_normal((5, 4, 8)), g.standard_normal((9, 4, 8)), g.standard_normal((9, 4, 8))
    out = A.attention(q, k, v, 4)[0]
    # a constant added to every score changes nothing, values enter linearly
    np.testing.assert_allclose(A.attention(q, k, 2 * v - 1, 4)[0], 2 * out - 1, rtol=1e-12)
    # a window of everything is none; the first token alone copies its value
    np.testing.assert_allclose(A.attention(q, k, v, 4, window=9)[0], out)
    np.testing.assert_allclose(A.attention(q[:1], k[:1], v[:1], 0)[0][0], v[0])
    # sinks that reach the window's first key are no mask
    np.testing.assert_allclose(A.attention(q, k, v, 4, window=2, sinks=8)[0], out)
    # zero queries average what they see
    np.testing.assert_allclose(A.attention(0 * q, k, v, 4, window=3)[0][0, 0], v[2:5, 0].mean(0))


def test_plan_by_hand():
    table = np.array([[5, -1, -1], [6, 7, -1], [-1, -1, -1]], np.int32)
    free = np.array([10, 11, 12, 13], np.int32)
    t, lens, slots, left = A.plan([3, 8, 0], [0, 2, 2, 7], table, free, 4, 4, 8)
    # request 0: 3 + 2 tokens in pages 5 and the topmost free one; 1 none; 2: 5 tokens in the next two
    assert t.tolist() == [[5, 13, -1], [6, 7, -1], [12, 11, -1]] and lens.tolist() == [5, 8, 5] and left == 1
    assert slots.tolist() == [23, 52, 48, 49, 50, 51, 44, -1]
    # too few pages: request 2 gets none
    t, lens, slots, left = A.plan([3, 8, 0], [0, 2, 2, 7], table, free, 2, 4, 8)
    assert lens.tolist() == [5, 8, 0] and left == 1 and slots.tolist() == [23, 44, -1, -1, -1, -1, -1, -1]
    l2, t2, f2, n2 = A.release([1, 0, 1], lens, t, free, left, 4)
    assert l2.tolist() == [0, 8, 0] and t2[0].tolist() == [-1, -1, -1] and n2 == 3 and f2[:3].tolist() == [10, 5, 11]
