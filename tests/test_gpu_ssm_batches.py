"""What the scan's bits depend on (GPU): not on whether the final state is
asked for, nor, with given segments, on the sequences beside one."""
import pytest
import torch

import gated_deltanet_02_amd as G
from tests import layer_util as U

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def run(e, lengths, final=True, **kw):
    fin = torch.empty(len(lengths), e["x"].shape[1], e["b"].shape[2], e["x"].shape[2], device="cuda") if final else None
    return G.gdn_ssm_prefill(e["x"], e["dt"], e["b"], e["c"], e["a_log"], e["dt_bias"], e["d_skip"], U.cu_of(lengths).cuda(),
                             e["init"], final_state=fin, **kw)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("P,H", [(128, 2), (64, 2), (64, 3), (32, 2)])
@pytest.mark.parametrize("seg", [-1, 0, 1])
def test_outputs_do_not_depend_on_the_final_state(dtype, P, H, seg):
    lengths = [300, 64, 0, 65, 31]
    e = U.to_gpu(U.scan_inputs(1, sum(lengths), H, 1, 64, P, dtype, len(lengths), init=True))
    assert torch.equal(run(e, lengths, True, segment_blocks=seg)[0], run(e, lengths, False, segment_blocks=seg)[0])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("P,H", [(128, 2), (64, 2), (16, 3)])
@pytest.mark.parametrize("seg", [-1, 1, 2])
def test_given_segments_make_sequences_independent(dtype, P, H, seg):
    lengths = [300, 64, 0, 65, 31, 129, 1]
    d = U.scan_inputs(2, sum(lengths), H, 1, 32, P, dtype, len(lengths), init=True)
    e = U.to_gpu(d)
    out, fin = run(e, lengths, segment_blocks=seg)
    start = 0
    for i, n in enumerate(lengths):
        one = {k: v if k in ("a_log", "dt_bias", "d_skip") else v[i: i + 1] if k == "init" else v[start: start + n]
               for k, v in e.items()}
        if n:
            o, f = run(one, [n], segment_blocks=seg)
            assert torch.equal(o, out[start: start + n]) and torch.equal(f[0], fin[i]), i
        start += n


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("packed", [True, False])
def test_one_pass_over_a_million_tokens(dtype, packed):
    """segment_blocks=-1 past 2^20 tokens: the bits of two calls, each one
    segment, with the state handed on."""
    half, T = 1 << 20, (1 << 20) + 1000
    g = torch.Generator(device="cuda").manual_seed(1)
    x, b, c = (torch.empty(T, 1, 16, dtype=dtype, device="cuda").normal_(generator=g) for _ in range(3))
    dt = 0.1 * torch.rand(T, 1, generator=g, device="cuda")
    cu = U.cu_of([T]).cuda() if packed else None
    fin, st = (torch.empty(1, 1, 16, 16, device="cuda") for _ in range(2))
    kw = dict(softplus=False, segment_blocks=-1)
    out, _ = G.gdn_ssm_prefill(x, dt, b, c, cu_seqlens=cu, final_state=fin, **kw)
    one, _ = G.gdn_ssm_prefill(x[:half], dt[:half], b[:half], c[:half], final_state=st, **kw)
    two, _ = G.gdn_ssm_prefill(x[half:], dt[half:], b[half:], c[half:], init_state=st, final_state=st, **kw)
    assert torch.equal(out[:half], one) and torch.equal(out[half:], two) and torch.equal(fin, st)
