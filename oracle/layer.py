"""Float64 references of the operators around a recurrent layer's
projections, from their definitions (numpy, token by token; test
infrastructure only).

``short_conv``: y[t] = bias + sum_j w[:, j] e[t + j] over a sequence's
history rows followed by its rows.  ``ssm_scan``: S <- a_t S + d_t b_t x_t^T,
y_t = S^T c_t + D x_t.  ``add_rms_norm``: r = x + residual,
y = r / sqrt(mean r^2 + eps) w, and its scales.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
SCALE_FLOOR = 2.0 ** -100


def softplus(x):
    return np.logaddexp(0.0, np.asarray(x, np.float64))


def silu(x):
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore"):
        return x / (1.0 + np.exp(-x))


def short_conv(x, w, bias=None, lengths=None, state_in=None, act=False):
    """x [T, D], w [D, W]; lengths per sequence (None: one); state_in
    [N, W - 1, D] or None.  Returns (y, state_out, magnitude), magnitude the
    same sum over absolute values (before the activation)."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    D, W = w.shape
    lengths = [x.shape[0]] if lengths is None else list(lengths)
    bias = np.zeros(D) if bias is None else np.asarray(bias, np.float64)
    y, mag = np.zeros_like(x), np.zeros_like(x)
    state = np.zeros((len(lengths), W - 1, D))
    t0 = 0
    for i, n in enumerate(lengths):
        hist = np.zeros((W - 1, D)) if state_in is None else np.asarray(state_in[i], np.float64)
        e = np.concatenate([hist, x[t0: t0 + n]])
        for t in range(n):
            y[t0 + t] = bias + sum(w[:, j] * e[t + j] for j in range(W))
            mag[t0 + t] = np.abs(bias) + sum(np.abs(w[:, j] * e[t + j]) for j in range(W))
        state[i] = e[n:]
        t0 += n
    return (silu(y) if act else y), state, mag


def ssm_scan(x, dt, b, c, a_log=None, dt_bias=None, d_skip=None, lengths=None, init=None,
             act=True):
    """x [T, H, P], dt [T, H], b, c [T, G, N], init [n_seq, H, N, P] or None.
    Returns (y [T, H, P], final [n_seq, H, N, P])."""
    x, dt, b, c = (np.asarray(v, np.float64) for v in (x, dt, b, c))
    T, H, P = x.shape
    G, N = b.shape[1:]
    lengths = [T] if lengths is None else list(lengths)
    zero = np.zeros(H)
    a_log, dt_bias, d_skip = (zero if v is None else np.asarray(v, np.float64)
                              for v in (a_log, dt_bias, d_skip))
    d = softplus(dt + dt_bias) if act else dt + dt_bias
    a = np.exp(-np.exp(a_log) * d)
    b, c = np.repeat(b, H // G, axis=1), np.repeat(c, H // G, axis=1)
    y = np.zeros_like(x)
    final = np.zeros((len(lengths), H, N, P))
    t0 = 0
    for i, n in enumerate(lengths):
        s = np.zeros((H, N, P)) if init is None else np.array(init[i], np.float64)
        for t in range(t0, t0 + n):
            s = a[t][:, None, None] * s + (d[t][:, None] * b[t])[:, :, None] * x[t][:, None, :]
            y[t] = np.einsum("hnp,hn->hp", s, c[t]) + d_skip[:, None] * x[t]
        final[i] = s
        t0 += n
    return y, final


def ssm_magnitude(x, dt, b, c, a_log=None, dt_bias=None, d_skip=None, lengths=None, init=None,
                  act=True):
    """The scan's sums over the absolute values of their terms (what rounding
    errors of its products scale with)."""
    ab = np.abs
    return ssm_scan(ab(x), dt, ab(b), ab(c), a_log, dt_bias, None if d_skip is None else ab(d_skip),
                    lengths, None if init is None else ab(init), act)


def add_rms_norm(x, residual=None, weight=None, eps=1e-6, group=0):
    """x [R, D].  Returns (r, y, scales): scales [R], or [R, ceil(D / group)]."""
    r = np.asarray(x, np.float64)
    if residual is not None:
        r = r + np.asarray(residual, np.float64)
    y = r / np.sqrt(np.mean(r * r, axis=1, keepdims=True) + eps)
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    top = np.abs(y)
    if group:
        n = -(-y.shape[1] // group)
        top = np.stack([top[:, g * group: (g + 1) * group].max(axis=1) for g in range(n)], axis=1)
    else:
        top = top.max(axis=1)
    return r, y, np.maximum(top, SCALE_FLOOR) / E4M3_MAX
