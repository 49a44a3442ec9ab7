"""The C ABI of the operators around the projections on the host: every
refusal with its status, before any HIP call (no GPU needed: descriptors
carry fake device addresses that are never dereferenced), the workspace
sizes, and the binding's structures against the header."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from gated_deltanet_02_amd import _binding as B
from gated_deltanet_02_amd import _layer as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL_ARG, DTYPE, SHAPE, LAYOUT, UNSUPPORTED, WORKSPACE, HIP = -1, -2, -3, -4, -5, -6, -7
BF16, F32, I32, I64, E4M3 = 1, 2, 3, 4, 5

_next = [0x100000000]


def fake(shape, dtype=BF16, addr=None, strides=None):
    """A descriptor with a fake device address of its own."""
    d = B.GdnTensor()
    if addr is None:
        addr = _next[0]
        _next[0] += 1 << 32
    d.data, d.dtype, d.ndim = addr, dtype, len(shape)
    acc, st = 1, []
    for s in reversed(shape):
        st.insert(0, acc)
        acc *= s
    for i, (s, t) in enumerate(zip(shape, strides or st)):
        d.shape[i], d.stride[i] = s, t
    return d


def ref(d):
    return ctypes.addressof(d) if isinstance(d, ctypes.Structure) else d


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.library_path()):
        pytest.fail("libgdn.so is not built (run __graft_entry__.build())")
    return L._functions()


def message():
    return B.lib().gdn_last_error().decode()


def expect(rc, want):
    assert rc == want, (rc, message())
    if want != 0:
        assert message()


# ---------------------------------------------------------------------------
# short convolution


def conv(lib, T=20, D=64, W=4, **kw):
    a = dict(x=fake((T, D)), w=fake((D, W), F32), bias=None, cu=None, si=None, so=None, out=fake((T, D)),
             flags=0)
    a.update(kw)
    return lib.gdn_short_conv(*[ref(a[k]) for k in ("x", "w", "bias", "cu", "si", "so", "out")], a["flags"], None)


def test_conv_refusals(lib):
    x = fake((20, 64))
    for kw, want in [
        (dict(x=None), NULL_ARG), (dict(w=None), NULL_ARG), (dict(out=None), NULL_ARG),
        (dict(x=fake((20, 64), I32), out=fake((20, 64), I32)), DTYPE), (dict(out=fake((20, 64), F32)), DTYPE),
        (dict(w=fake((64, 4), BF16)), DTYPE), (dict(flags=2), SHAPE),
        (dict(x=fake((20,)), out=fake((20,))), SHAPE), (dict(out=fake((21, 64))), SHAPE),
        (dict(w=fake((63, 4), F32)), SHAPE), (dict(w=fake((64, 5), F32)), SHAPE), (dict(w=fake((64, 0), F32)), SHAPE),
        (dict(w=fake((64, 4), F32, strides=(8, 1))), LAYOUT),
        (dict(x=fake((20, 64), strides=(128, 2))), LAYOUT), (dict(x=fake((20, 64), strides=(-64, 1))), LAYOUT),
        (dict(x=fake((20, 64), addr=0)), NULL_ARG), (dict(x=fake((20, 64), addr=0x1001)), LAYOUT),
        (dict(bias=0x1002), LAYOUT),
        (dict(out=fake((20, 64), strides=(32, 1))), LAYOUT),                     # rows overlap
        (dict(x=x, out=fake((20, 64), addr=x.data)), LAYOUT),                     # in place
        (dict(x=x, out=fake((20, 64), addr=x.data + 128)), LAYOUT),               # one row behind
        (dict(cu=fake((3,), F32)), DTYPE), (dict(cu=fake((1,), I32)), SHAPE),
        (dict(cu=fake((3,), I32, strides=(2,))), LAYOUT), (dict(cu=fake((3,), I32, addr=0)), NULL_ARG),
        (dict(cu=fake((3,), I64, addr=0x1004)), LAYOUT),
        (dict(x=fake((2, 10, 64)), out=fake((2, 10, 64)), cu=fake((3,), I32)), SHAPE),
        (dict(x=fake((2, 10, 64), strides=(1280, 64, 1)), out=fake((2, 10, 64))), LAYOUT),
        (dict(x=fake((0, 5, 64)), out=fake((0, 5, 64))), SHAPE),
        (dict(si=fake((1, 3, 64), F32)), DTYPE), (dict(si=fake((2, 3, 64))), SHAPE), (dict(so=fake((1, 2, 64))), SHAPE),
        (dict(si=fake((1, 3, 64), strides=(192, 65, 1))), LAYOUT), (dict(so=fake((1, 3, 64), addr=0)), NULL_ARG),
    ]:
        expect(conv(lib, **kw), want)
    st = fake((1, 3, 64))
    expect(conv(lib, si=st, so=fake((1, 3, 64), addr=st.data + 128)), LAYOUT)
    expect(conv(lib, x=x, so=fake((1, 3, 64), addr=x.data)), LAYOUT)
    expect(conv(lib, si=st, so=st, out=fake((20, 64), addr=st.data)), LAYOUT)
    expect(conv(lib, x=fake((1 << 31, 64)), out=fake((1 << 31, 64))), SHAPE)


# ---------------------------------------------------------------------------
# the scan


def opts(**kw):
    o = L.GdnSsmOptions()
    o.flags = 1
    for k, v in kw.items():
        setattr(o, k, v)
    return o


def scan(lib, T=100, H=4, G=2, N=64, P=32, ws=(0x10000, 1 << 22), **kw):
    a = dict(x=fake((T, H, P)), dt=fake((T, H), F32), b=fake((T, G, N)), c=fake((T, G, N)), cu=None,
             init=None, out=fake((T, H, P)), fin=None, opts=None)
    a.update(kw)
    return lib.gdn_ssm_prefill(*[ref(a[k]) for k in ("x", "dt", "b", "c", "cu", "init", "out", "fin", "opts")], ws[0],
                               ws[1], None)


def test_scan_refusals(lib):
    x, s = fake((100, 4, 32)), (100, 4, 32)
    for kw, want in [
        *[({k: None}, NULL_ARG) for k in ("x", "dt", "b", "c", "out")],
        (dict(x=fake(s, I32)), DTYPE), (dict(b=fake((100, 2, 64), F32)), DTYPE), (dict(c=fake((100, 2, 64), F32)), DTYPE),
        (dict(out=fake(s, F32)), DTYPE), (dict(dt=fake((100, 4), BF16)), DTYPE),
        (dict(x=fake((100, 4))), SHAPE), (dict(b=fake((1, 100, 2, 64))), SHAPE), (dict(c=fake((100, 2, 32))), SHAPE),
        (dict(b=fake((99, 2, 64)), c=fake((99, 2, 64))), SHAPE), (dict(out=fake((100, 4, 64))), SHAPE),
        (dict(dt=fake((100, 3), F32)), SHAPE), (dict(dt=fake((1, 100, 4), F32)), SHAPE),
        (dict(b=fake((100, 3, 64)), c=fake((100, 3, 64))), SHAPE), (dict(b=fake((100, 0, 64)), c=fake((100, 0, 64))), SHAPE),
        (dict(b=fake((100, 2, 48)), c=fake((100, 2, 48))), UNSUPPORTED), (dict(x=fake((100, 4, 256)), out=fake((100, 4, 256))), UNSUPPORTED),
        (dict(x=fake(s, strides=(128, 32, 2))), LAYOUT), (dict(x=fake(s, strides=(132, 32, 1))), LAYOUT),
        (dict(c=fake((100, 2, 64), addr=0x10008)), LAYOUT), (dict(b=fake((100, 2, 64), addr=0)), NULL_ARG),
        (dict(out=fake(s, strides=(64, 32, 1))), LAYOUT), (dict(out=fake(s, strides=(0, 32, 1))), LAYOUT),
        (dict(x=fake(s, strides=(1 << 25, 32, 1))), LAYOUT),
        (dict(dt=fake((100, 4), F32, strides=(1 << 25, 1))), LAYOUT),
        (dict(dt=fake((100, 4), F32, addr=0x1002)), LAYOUT),
        (dict(init=fake((1, 4, 64, 32), BF16)), DTYPE), (dict(init=fake((2, 4, 64, 32), F32)), SHAPE),
        (dict(fin=fake((1, 4, 32, 64), F32)), SHAPE), (dict(fin=fake((1, 4, 64, 32), F32, addr=0x1008)), LAYOUT),
        (dict(fin=fake((1, 4, 64, 32), F32, strides=(8192, 2048, 33, 1))), LAYOUT),
        (dict(cu=fake((2,), F32)), DTYPE), (dict(cu=fake((2, 2), I32)), SHAPE),
        (dict(opts=opts(flags=2)), SHAPE), (dict(opts=opts(segment_blocks=-2)), SHAPE), (dict(opts=opts(a_log=0x1001)), LAYOUT),
        (dict(x=x, out=fake(s, addr=x.data)), LAYOUT),
        (dict(ws=(None, 0), opts=opts(segment_blocks=1)), WORKSPACE), (dict(ws=(0x10000, 64), cu=fake((3,), I32)), WORKSPACE),
        (dict(ws=(0x10010, 1 << 40)), WORKSPACE),
    ]:
        expect(scan(lib, **kw), want)
    st = fake((1, 4, 64, 32), F32)
    expect(scan(lib, init=st, fin=fake((1, 4, 64, 32), F32, addr=st.data + 4096)), LAYOUT)
    expect(scan(lib, x=x, fin=fake((1, 4, 64, 32), F32, addr=x.data)), LAYOUT)
    ws = fake((1 << 20,), F32)
    expect(scan(lib, x=fake(s, addr=ws.data), ws=(ws.data, 1 << 22), opts=opts(segment_blocks=1)), LAYOUT)
    expect(scan(lib, H=65536, G=1, P=16, N=16, T=1), UNSUPPORTED)


def wsize(lib, T, H, G, N, P, cu=None, o=None, dt=BF16):
    n = ctypes.c_size_t(0)
    x, b = fake((T, H, P), dt), fake((T, G, N), dt)
    expect(lib.gdn_ssm_workspace_size(ref(x), ref(b), ref(cu), ref(o), ctypes.byref(n)), 0)
    return n.value


def test_scan_workspace(lib):
    assert wsize(lib, 100, 4, 2, 64, 32) == 0                      # a short sequence: one pass
    assert wsize(lib, 100000, 4, 2, 64, 32, o=opts(segment_blocks=-1)) == 0
    # segments of one block: a decay and a state per segment and head, and the
    # end of each sequence and head
    got = wsize(lib, 640, 4, 2, 64, 32, o=opts(segment_blocks=1))
    assert got == 256 + (10 + 1) * 4 * 64 * 32 * 4
    # packed: the table and the segments' offsets besides
    got = wsize(lib, 640, 4, 2, 64, 32, cu=fake((4,), I32), o=opts(segment_blocks=-1))
    assert got == 256 + 256
    n = ctypes.c_size_t(0)
    x, b = fake((10, 4, 32)), fake((10, 2, 64))
    expect(lib.gdn_ssm_workspace_size(None, ref(b), None, None, ctypes.byref(n)), NULL_ARG)
    expect(lib.gdn_ssm_workspace_size(ref(x), ref(b), None, None, None), NULL_ARG)


# ---------------------------------------------------------------------------
# the step


def step(lib, n=3, H=4, G=2, N=64, P=32, **kw):
    a = dict(x=fake((n, H, P)), dt=fake((n, H), F32), b=fake((n, G, N)), c=fake((n, G, N)),
             state=fake((n, H, N, P), F32), out=fake((n, H, P)), opts=None)
    a.update(kw)
    return lib.gdn_ssm_decode(*[ref(a[k]) for k in ("x", "dt", "b", "c", "state", "out", "opts")], None)


def test_step_refusals(lib):
    x, s = fake((3, 4, 32)), (3, 4, 32)
    for kw, want in [
        *[({k: None}, NULL_ARG) for k in ("x", "dt", "b", "c", "state", "out")],
        (dict(x=fake(s, I32)), DTYPE), (dict(c=fake((3, 2, 64), F32)), DTYPE), (dict(state=fake((3, 4, 64, 32), BF16)), DTYPE),
        (dict(dt=fake((3, 4), BF16)), DTYPE), (dict(x=fake((1, 3, 4, 32))), SHAPE), (dict(b=fake((2, 2, 64)), c=fake((2, 2, 64))), SHAPE),
        (dict(state=fake((2, 4, 64, 32), F32)), SHAPE), (dict(dt=fake((3, 5), F32)), SHAPE),
        (dict(b=fake((3, 3, 64)), c=fake((3, 3, 64))), SHAPE), (dict(b=fake((3, 2, 8)), c=fake((3, 2, 8))), UNSUPPORTED),
        (dict(state=fake((3, 4, 64, 32), F32, addr=0x1004)), LAYOUT), (dict(x=fake(s, addr=0x1002)), LAYOUT),
        (dict(x=fake(s, strides=(130, 32, 1))), LAYOUT), (dict(out=fake(s, strides=(128, 0, 1))), LAYOUT),
        (dict(x=x, out=fake(s, addr=x.data)), LAYOUT), (dict(opts=opts(flags=4)), SHAPE),
    ]:
        expect(step(lib, **kw), want)
    st = fake((3, 4, 64, 32), F32)
    expect(step(lib, state=st, x=fake(s, addr=st.data + 64)), LAYOUT)
    expect(step(lib, n=0, x=fake((0, 4, 32), addr=0), b=fake((0, 2, 64), addr=0), c=fake((0, 2, 64), addr=0),
                dt=fake((0, 4), F32, addr=0), state=fake((0, 4, 64, 32), F32, addr=0), out=fake((0, 4, 32), addr=0)), 0)


# ---------------------------------------------------------------------------
# the residual norm


def norm(lib, R=5, D=256, eps=1e-6, **kw):
    a = dict(x=fake((R, D)), r=None, w=None, ro=None, out=fake((R, D)), q=None, s=None)
    a.update(kw)
    return lib.gdn_add_rms_norm(ref(a["x"]), ref(a["r"]), a["w"], eps, ref(a["ro"]), ref(a["out"]), ref(a["q"]),
                                ref(a["s"]), None)


def test_norm_refusals(lib):
    x, r, s = fake((5, 256)), fake((5, 256)), (5, 256)
    q, sc = fake(s, E4M3), fake((5,), F32)
    for kw, want in [
        (dict(x=None), NULL_ARG), (dict(out=None), NULL_ARG), (dict(q=q), NULL_ARG), (dict(s=sc), NULL_ARG),
        (dict(x=fake(s, I32)), DTYPE), (dict(r=fake(s, F32)), DTYPE), (dict(ro=fake(s, F32)), DTYPE), (dict(out=fake(s, F32)), DTYPE),
        (dict(q=fake(s, BF16), s=sc), DTYPE), (dict(q=q, s=fake((5,), BF16)), DTYPE), (dict(x=fake(s, 9)), DTYPE),
        (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(w=0x1002), LAYOUT),
        (dict(x=fake((5, 2, 128))), SHAPE), (dict(r=fake((4, 256))), SHAPE), (dict(out=fake((5, 255))), SHAPE),
        (dict(q=q, s=fake((4,), F32)), SHAPE), (dict(q=q, s=fake((5, 3), F32)), SHAPE),
        (dict(q=q, s=fake((5, 2), F32, strides=(4, 1))), LAYOUT),
        (dict(x=fake((5, 65537)), out=fake((5, 65537))), UNSUPPORTED), (dict(x=fake((5, 0)), out=fake((5, 0))), UNSUPPORTED),
        (dict(x=fake(s, strides=(512, 2))), LAYOUT), (dict(x=fake(s, addr=0)), NULL_ARG), (dict(out=fake(s, strides=(128, 1))), LAYOUT),
        (dict(x=x, out=fake(s, addr=x.data + 512)), LAYOUT), (dict(x=x, out=fake(s, addr=x.data, strides=(512, 1))), LAYOUT),
        (dict(r=r, ro=fake(s, addr=r.data + 16)), LAYOUT), (dict(x=x, q=fake(s, E4M3, addr=x.data), s=sc), LAYOUT),
        (dict(ro=r, out=r), LAYOUT), (dict(q=q, s=fake((5,), F32, addr=q.data)), LAYOUT),
        (dict(x=fake(s, F32, addr=x.data), out=fake(s, F32, addr=x.data + 4)), LAYOUT),
    ]:
        expect(norm(lib, **kw), want)
    w = fake((256,), F32)
    expect(norm(lib, w=w.data, out=fake(s, addr=w.data)), LAYOUT)
    expect(norm(lib, R=0, x=fake((0, 256), addr=0), out=fake((0, 256), addr=0)), 0)


# ---------------------------------------------------------------------------
# the header and the binding


def test_counts_at_the_limits(lib):
    """Counts that a kernel's 32-bit counters could run past are refused."""
    most = (1 << 31) - (1 << 21)
    at = dict(bias=None, x=fake((most + 1, 8)), out=fake((most + 1, 8), addr=1 << 44))
    expect(conv(lib, D=8, **at), SHAPE)
    assert "2^31 - 2^21" in message()
    expect(conv(lib, x=fake((1, most + 1)), out=fake((1, most + 1)), w=fake((most + 1, 4), F32, addr=1 << 44)), SHAPE)
    expect(conv(lib, cu=fake((most + 2,), I32)), SHAPE)
    n = ctypes.c_size_t(0)
    # launches of 2^32 threads: 4 P per segment and head in the scan, 256 per
    # sequence and head where segments are joined
    cut = opts(segment_blocks=1)
    for T, H, P, n_seq, o, want in [
            (most + 1, 1, 16, None, None, SHAPE), (most, 1, 16, None, None, 0), (100, 1, 16, most + 1, None, SHAPE),
            (4096, 4000, 64, 4180, None, 0), (4096, 4000, 64, 4190, None, SHAPE),
            (4096, 4000, 16, 4190, cut, 0), (4096, 4000, 16, 4195, cut, SHAPE), (4096, 4000, 16, 4195, None, 0)]:
        x, b = fake((T, H, P)), fake((T, 1, 16))
        cu = None if n_seq is None else fake((n_seq + 1,), I32)
        expect(lib.gdn_ssm_workspace_size(ref(x), ref(b), ref(cu), ref(o), ctypes.byref(n)), want)


def test_options_struct_matches_the_header(tmp_path):
    src = tmp_path / "l.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "gdn.h"\nint main(void) {\n'
                   '  printf("%zu", sizeof(gdn_ssm_options));\n' +
                   "".join(f'  printf(" %zu", offsetof(gdn_ssm_options, {f}));\n' for f, _ in L.GdnSsmOptions._fields_) +
                   "  return 0;\n}\n")
    exe = tmp_path / "l"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", f"-I{ROOT}/include", str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(L.GdnSsmOptions)] + [getattr(L.GdnSsmOptions, f).offset for f, _ in L.GdnSsmOptions._fields_]


def test_constants_match_the_header(lib):
    src = open(os.path.join(ROOT, "include", "gdn.h")).read()
    for name, value in (("GDN_SSM_SOFTPLUS", L.SSM_SOFTPLUS), ("GDN_CONV_SILU", L.CONV_SILU), ("GDN_E4M3", L.E4M3)):
        assert int(re.search(rf"#define {name} (\d+)u?\b", src).group(1)) == value
    o = L.gdn_ssm_default_options()
    assert (o.a_log, o.dt_bias, o.d_skip, o.flags, o.segment_blocks) == (None, None, None, L.SSM_SOFTPLUS, 0)


def test_binding_refuses_cpu_tensors():
    import gated_deltanet_02_amd as G
    x = torch.randn(4, 64)
    for call in (lambda: G.gdn_short_conv(x, torch.randn(64, 4)), lambda: G.gdn_add_rms_norm(x),
                 lambda: G.gdn_ssm_prefill(x.view(4, 4, 16), x[:, :4], x.view(4, 4, 16), x.view(4, 4, 16)),
                 lambda: G.gdn_ssm_decode(x.view(4, 4, 16), x[:, :4], x.view(4, 4, 16), x.view(4, 4, 16), torch.zeros(4, 4, 16, 16))):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
