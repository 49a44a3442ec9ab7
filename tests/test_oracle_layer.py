"""The float64 references of the operators around the projections against
closed forms and independent evaluations (CPU)."""
import numpy as np
import pytest

from oracle import gates, layer


def rng(seed=0):
    return np.random.Generator(np.random.PCG64(seed))


def test_short_conv_against_numpy_convolve():
    r = rng()
    x, w, h = r.normal(size=(11, 3)), r.normal(size=(3, 4)), r.normal(size=(2, 3, 3))
    y, state, _ = layer.short_conv(x, w, lengths=[7, 4], state_in=h)
    for i, (lo, hi) in enumerate([(0, 7), (7, 11)]):
        e = np.concatenate([h[i], x[lo:hi]])
        for ch in range(3):
            np.testing.assert_allclose(y[lo:hi, ch], np.convolve(e[:, ch], w[ch, ::-1], "valid"))
        np.testing.assert_array_equal(state[i], e[-3:])


def test_short_conv_agrees_with_the_fused_reference():
    r = rng(1)
    x, w, h = r.normal(size=(9, 5)), r.normal(size=(5, 4)), r.normal(size=(2, 3, 5))
    y, state, _ = layer.short_conv(x, w, lengths=[2, 7], state_in=h, act=True)
    want, want_state = gates.short_conv(x, w, lengths=[2, 7], state=h)
    np.testing.assert_allclose(y, gates.silu(want))
    np.testing.assert_array_equal(state, want_state)


def test_short_conv_bias_and_one_tap():
    x = rng(2).normal(size=(4, 2))
    y, state, _ = layer.short_conv(x, np.array([[2.0], [-1.0]]), bias=[1.0, 0.5])
    np.testing.assert_allclose(y, x * [2.0, -1.0] + [1.0, 0.5])
    assert state.shape == (1, 0, 2)


def test_ssm_scan_as_an_explicit_sum():
    """y_i = sum_j (c_i . b_j) prod_{j < s <= i} a_s d_j x_j + D x_i + c_i^T prod a S0."""
    r = rng(3)
    T, H, G, N, P = 6, 4, 2, 3, 2
    x, dt = r.normal(size=(T, H, P)), r.normal(size=(T, H))
    b, c = r.normal(size=(T, G, N)), r.normal(size=(T, G, N))
    al, bias, skip = r.normal(size=H), r.normal(size=H), r.normal(size=H)
    init = r.normal(size=(1, H, N, P))
    y, final = layer.ssm_scan(x, dt, b, c, al, bias, skip, init=init)
    d = np.log1p(np.exp(dt + bias))
    a = np.exp(-np.exp(al) * d)
    for h in range(H):
        g = h // 2
        for i in range(T):
            want = skip[h] * x[i, h] + np.prod(a[: i + 1, h]) * c[i, g] @ init[0, h]
            for j in range(i + 1):
                want = want + (c[i, g] @ b[j, g]) * np.prod(a[j + 1: i + 1, h]) * d[j, h] * x[j, h]
            np.testing.assert_allclose(y[i, h], want, rtol=1e-12, atol=1e-12)
        want = np.prod(a[:, h]) * init[0, h]
        for j in range(T):
            want = want + np.prod(a[j + 1:, h]) * d[j, h] * np.outer(b[j, g], x[j, h])
        np.testing.assert_allclose(final[0, h], want, rtol=1e-12, atol=1e-12)


def test_ssm_scan_is_linear_attention_without_decay():
    """d = 1 and a rate of e^-60 (no decay): cumulative sums of b x^T."""
    r = rng(4)
    x, b, c = r.normal(size=(5, 1, 2)), r.normal(size=(5, 1, 3)), r.normal(size=(5, 1, 3))
    y, final = layer.ssm_scan(x, np.ones((5, 1)), b, c, a_log=[-60.0], act=False)
    sums = np.cumsum(b[:, 0, :, None] * x[:, 0, None, :], axis=0)
    np.testing.assert_allclose(y[:, 0], np.einsum("tnp,tn->tp", sums, c[:, 0]))
    np.testing.assert_allclose(final[0, 0], sums[-1])


def test_ssm_scan_continues_and_packs():
    r = rng(5)
    x, dt = r.normal(size=(8, 2, 2)), r.normal(size=(8, 2))
    b, c = r.normal(size=(8, 1, 3)), r.normal(size=(8, 1, 3))
    whole, end = layer.ssm_scan(x, dt, b, c)
    one, mid = layer.ssm_scan(x[:3], dt[:3], b[:3], c[:3])
    two, end2 = layer.ssm_scan(x[3:], dt[3:], b[3:], c[3:], init=mid)
    np.testing.assert_allclose(np.concatenate([one, two]), whole)
    np.testing.assert_allclose(end2, end)
    packed, ends = layer.ssm_scan(x, dt, b, c, lengths=[3, 0, 5])
    np.testing.assert_allclose(packed[:3], one)
    np.testing.assert_allclose(ends[0], mid[0])
    assert not ends[1].any()
    np.testing.assert_allclose(packed[3:], layer.ssm_scan(x[3:], dt[3:], b[3:], c[3:])[0])


@pytest.mark.parametrize("group", [0, 2])
def test_add_rms_norm_by_hand(group):
    """r = (3, 4, 0, 0): mean square 25/4, y = r / 2.5 (eps 0)."""
    r, y, s = layer.add_rms_norm([[1.0, 4.0, -1.0, 0.0]], [[2.0, 0.0, 1.0, 0.0]], eps=0.0, group=group)
    np.testing.assert_array_equal(r, [[3.0, 4.0, 0.0, 0.0]])
    np.testing.assert_allclose(y, [[1.2, 1.6, 0.0, 0.0]])
    want = [[1.6 / 448, 2.0 ** -100 / 448]] if group else [1.6 / 448]
    np.testing.assert_allclose(s, want)
