"""Inputs, derived tolerances and checks of the tests of the operators around
the projections (not collected by pytest).

Tolerances.  A rounding to a type costs at most half a step,
``HALF[dtype]`` relative to the value.  What the fp32 arithmetic costs
scales with the sum M of the absolute values of a result's terms:

* convolution: at most five terms and the activation, a few 2^-24 each:
  2^-20 (M + 1) (silu's slope is below 1.1);
* scan outputs: M_ij and the state enter their products as two bf16 terms,
  each term within 2^-8 of what it rounds, so within 2^-16 of a product
  together; sums of up to 128 + 64 + 128 fp32 terms and decays from sums of
  up to 64 rounded logarithms add less than 2^-15: 2^-14 M;
* scan states: three terms (2^-24), sums of 64 terms per block carried over
  64 blocks, the same decays: 2^-15 M;
* step: fp32 products and sums of up to 128 terms, exp of a rounded
  exponent of up to about 20: 2^-17 M;
* norm: the sum of squares of positive terms, at most about 100 in a row on
  one thread and then a tree: 2^-17 relative.
"""
from __future__ import annotations

import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24, torch.float8_e4m3fn: 2.0 ** -4}
CONV_F32, SCAN_OUT, SCAN_STATE, STEP_F32, NORM_F32 = 2.0 ** -20, 2.0 ** -14, 2.0 ** -15, 2.0 ** -17, 2.0 ** -17


def f64(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g).to(dtype)


def cu_of(lengths, dtype=torch.int32):
    return torch.tensor([0] + list(np.cumsum(lengths)), dtype=dtype)


def check(got, want, bound, label):
    """Every element within its bound of the reference."""
    got = f64(got) if isinstance(got, torch.Tensor) else got
    want, bound = np.asarray(want), np.asarray(bound)
    assert got.shape == want.shape, (label, got.shape, want.shape)
    assert np.isfinite(got).all(), f"{label}: not finite"
    err = np.abs(got - want)
    over = err / np.maximum(bound, 1e-300)
    worst = float(over.max()) if over.size else 0.0
    print(f"  {label}: max error {float(err.max()) if err.size else 0.0:.3e}, {worst:.3f} of its bound", flush=True)
    assert worst <= 1.0, f"{label}: {worst:.3f} of the bound at {np.unravel_index(over.argmax(), over.shape)}"


def scan_inputs(seed, T, H, G, N, P, dtype, n_seq, init=False):
    """CPU inputs as a layer produces them: steps of about 1e-3 .. 1, rates
    1 .. 16."""
    g = gen(seed)
    d = dict(x=randn(g, T, H, P, dtype=dtype), dt=randn(g, T, H), b=randn(g, T, G, N, dtype=dtype),
             c=randn(g, T, G, N, dtype=dtype))
    d["a_log"] = torch.log(1 + 15 * torch.rand(H, generator=g))
    d["dt_bias"] = -6.9 + 4.6 * torch.rand(H, generator=g)
    d["d_skip"] = 1 + 0.1 * randn(g, H)
    d["init"] = 0.5 * randn(g, n_seq, H, N, P) if init else None
    return d


def to_gpu(d):
    return {k: None if v is None else v.cuda() for k, v in d.items()}
