"""Seeded configurations of the scan against float64 (GPU): types, head sizes
and groups, batches packed or not with empty and one-token sequences, segments,
states in and out, steps and rates, strided rows."""
import random

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


def lengths_of(r):
    kind = r.random()
    if kind < 0.25:
        return [r.randint(1, 600)], False
    if kind < 0.4:
        return [r.randint(1, 200)] * r.randint(2, 6), False
    n = r.choice([2, 5, 20, 70])
    return [r.choice([0, 1, 31, 32, 33, 63, 64, 65, 127, 129, r.randint(0, 400 if n < 20 else 60)]) for _ in range(n)] + [r.randint(1, 300)], True


@pytest.mark.parametrize("seed", range(80))
def test_scan_sweep(seed):
    r = random.Random(seed)
    dtype = r.choice([BF16, BF16, F32])
    lengths, packed = lengths_of(r)
    T, n = sum(lengths), len(lengths)
    g = r.choice([1, 2, 3])
    H, N, P = g * r.choice([1, 2, 3, 4]), r.choice([16, 32, 64, 128]), r.choice([16, 32, 64, 128])
    init, final, seg = r.random() < 0.6, r.random() < 0.8, r.choice([0, 0, -1, 1, 2, 3])
    d = U.scan_inputs(seed, T, H, g, N, P, dtype, n, init=init)
    if r.random() < 0.3:  # large steps among the others
        d["dt"] = torch.where(torch.rand(T, H, generator=U.gen(seed)) < 0.05, torch.tensor(float(r.choice([10, 60, 300]))), d["dt"])
    if r.random() < 0.2:
        d["dt_bias"] = None
    if r.random() < 0.2:
        d["d_skip"] = None
    e = U.to_gpu(d)
    label = f"{dtype} T={T} n={n} H={H}/{g} {N}x{P} packed={packed} init={init} final={final} segments={seg}"
    print(label, flush=True)
    if r.random() < 0.5:
        rows = torch.cat([e["x"].flatten(1), e["b"].flatten(1), e["c"].flatten(1)], 1).contiguous()
        e["x"] = rows[:, : H * P].view(T, H, P)
        e["b"] = rows[:, H * P: H * P + g * N].view(T, g, N)
        e["c"] = rows[:, H * P + g * N:].view(T, g, N)
    wide = torch.full((T, H, 2 * P), 3.0, dtype=dtype, device="cuda")
    out = wide[:, :, P:]
    fin = torch.full((n, H, N, P), 7.0, device="cuda") if final else None
    args, cu, o = [e[k] for k in ("x", "dt", "b", "c")], None, out
    if packed:
        cu = U.cu_of(lengths, r.choice([torch.int32, torch.int64])).cuda()
    elif n > 1:
        args = [v.unflatten(0, (n, lengths[0])) for v in args]
        o = out.unflatten(0, (n, lengths[0]))
    if init and final and r.random() < 0.5:
        fin = e["init"]
    G.gdn_ssm_prefill(*args, e["a_log"], e["dt_bias"], e["d_skip"], cu, e["init"], o, fin, segment_blocks=seg)
    a = [U.f64(d[k]) for k in ("x", "dt", "b", "c", "a_log", "dt_bias", "d_skip")]
    y, s = layer.ssm_scan(*a, lengths=lengths, init=U.f64(d["init"]))
    my, ms = layer.ssm_magnitude(*a, lengths=lengths, init=U.f64(d["init"]))
    U.check(out, y, U.HALF[dtype] * np.abs(y) + U.SCAN_OUT * my + 2.0 ** -100, label + " out")
    if final:
        U.check(fin, s, U.SCAN_STATE * ms + 2.0 ** -100, label + " state")
    assert (wide[:, :, :P] == 3).all()
