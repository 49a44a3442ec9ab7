"""The C ABI of the attention over a paged cache on the host: every refusal
with its status, before any HIP call (no GPU needed: descriptors carry fake
device addresses that are never dereferenced), the workspace sizes, and the
binding's structures against the header."""
import ctypes
import os
import subprocess

import pytest
import torch

from gated_deltanet_02_amd import _attn as T
from gated_deltanet_02_amd import _binding as B
from tests.test_layer_boundary import (BF16, DTYPE, F32, I32, I64, LAYOUT, NULL_ARG, ROOT, SHAPE, UNSUPPORTED, WORKSPACE, expect, fake,
                                       message, ref)

MOST = (1 << 31) - (1 << 21)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.library_path()):
        pytest.fail("libgdn.so is not built (run __graft_entry__.build())")
    return T._functions()


def options(scale=0.0, window=0, sinks=0):
    o = T.gdn_attn_default_options()
    o.scale, o.window, o.sinks = scale, window, sinks
    return o


# ---------------------------------------------------------------------------
# plan and release


def plan(lib, N=3, width=8, t=12, page=16, **kw):
    a = dict(ctx=fake((N,), I32), cu=fake((N + 1,), I32), table=fake((N, width), I32), free=fake((30,), I32), n_free=fake((1,), I32),
             lens=fake((N,), I32), slots=fake((t,), I64), left=fake((1,), I32), page=page)
    a.update(kw)
    return lib.gdn_cache_plan(*[ref(a[k]) for k in ("ctx", "cu", "table", "free", "n_free")], a["page"],
                              *[ref(a[k]) for k in ("lens", "slots", "left")], None)


def test_plan_refusals(lib):
    ctx, free, table = fake((3,), I32), fake((30,), I32), fake((3, 8), I32)
    for kw, want in [
        *[({k: None}, NULL_ARG) for k in ("ctx", "table", "free", "n_free", "lens", "slots", "left")],
        *[({k: fake(s, I64)}, DTYPE) for k, s in (("ctx", (3,)), ("table", (3, 8)), ("free", (30,)), ("n_free", (1,)), ("lens", (3,)),
                                                   ("left", (1,)))],
        (dict(slots=fake((12,), I32)), DTYPE), (dict(cu=fake((4,), F32)), DTYPE),
        (dict(ctx=fake((3, 1), I32)), SHAPE), (dict(table=fake((4, 8), I32)), SHAPE), (dict(table=fake((24,), I32)), SHAPE),
        (dict(lens=fake((4,), I32)), SHAPE), (dict(n_free=fake((2,), I32)), SHAPE), (dict(left=fake((2,), I32)), SHAPE),
        (dict(cu=fake((5,), I32)), SHAPE), (dict(cu=None), SHAPE), (dict(page=0), SHAPE), (dict(page=-16), SHAPE),
        (dict(page=1 << 30), SHAPE), (dict(slots=fake((MOST + 1,), I64)), SHAPE),
        (dict(ctx=fake((3,), I32, strides=(2,))), LAYOUT), (dict(table=fake((3, 8), I32, strides=(16, 2))), LAYOUT),
        (dict(table=fake((3, 8), I32, strides=(4, 1))), LAYOUT), (dict(free=fake((30,), I32, strides=(-1,))), LAYOUT),
        (dict(ctx=fake((3,), I32, addr=0)), NULL_ARG),
        # an output over an input, or over another output
        (dict(ctx=ctx, lens=fake((3,), I32, addr=ctx.data + 4)), LAYOUT), (dict(free=free, table=fake((3, 8), I32, addr=free.data)), LAYOUT),
        (dict(free=free, left=fake((1,), I32, addr=free.data + 8)), LAYOUT), (dict(table=table, slots=fake((12,), I64, addr=table.data)), LAYOUT),
    ]:
        expect(plan(lib, **kw), want)
    n = (1 << 20) + 1
    expect(plan(lib, N=n, ctx=fake((n,), I32)), SHAPE)


def release(lib, N=3, width=8, page=16, **kw):
    a = dict(done=fake((N,), I32), lens=fake((N,), I32), table=fake((N, width), I32), free=fake((30,), I32), n_free=fake((1,), I32), page=page)
    a.update(kw)
    return lib.gdn_cache_release(*[ref(a[k]) for k in ("done", "lens", "table", "free", "n_free")], a["page"], None)


def test_release_refusals(lib):
    done, free = fake((3,), I32), fake((30,), I32)
    for kw, want in [
        *[({k: None}, NULL_ARG) for k in ("done", "lens", "table", "free", "n_free")],
        *[({k: fake(s, I64)}, DTYPE) for k, s in (("done", (3,)), ("lens", (3,)), ("table", (3, 8)), ("free", (30,)), ("n_free", (1,)))],
        (dict(lens=fake((2,), I32)), SHAPE), (dict(table=fake((2, 8), I32)), SHAPE), (dict(n_free=fake((0,), I32)), SHAPE),
        (dict(page=0), SHAPE), (dict(table=fake((3, 8), I32, strides=(0, 1))), LAYOUT),
        (dict(done=done, lens=fake((3,), I32, addr=done.data)), LAYOUT), (dict(free=free, n_free=fake((1,), I32, addr=free.data)), LAYOUT),
    ]:
        expect(release(lib, **kw), want)
    expect(release(lib, N=0, done=fake((0,), I32, addr=0), lens=fake((0,), I32, addr=0), table=fake((0, 8), I32, addr=0)), 0)


# ---------------------------------------------------------------------------
# store


def store(lib, t=5, kv=2, d=128, pages=7, page=16, dtype=BF16, **kw):
    a = dict(k=fake((t, kv, d), dtype), v=fake((t, kv, d), dtype), slots=fake((t,), I64), kc=fake((pages, page, kv, d), dtype),
             vc=fake((pages, page, kv, d), dtype))
    a.update(kw)
    return lib.gdn_cache_store(*[ref(a[k]) for k in ("k", "v", "slots", "kc", "vc")], None)


def test_store_refusals(lib):
    s, c = (5, 2, 128), (7, 16, 2, 128)
    k, kc = fake(s), fake(c)
    for kw, want in [
        *[({n: None}, NULL_ARG) for n in ("k", "v", "slots", "kc", "vc")],
        (dict(dtype=I32), DTYPE), (dict(v=fake(s, F32)), DTYPE), (dict(kc=fake(c, F32)), DTYPE), (dict(vc=fake(c, F32)), DTYPE),
        (dict(slots=fake((5,), I32)), DTYPE), (dict(slots=fake((4,), I64)), SHAPE), (dict(v=fake((5, 2, 64))), SHAPE),
        (dict(v=fake((4, 2, 128))), SHAPE), (dict(vc=fake((8, 16, 2, 128))), SHAPE), (dict(k=fake((5, 256))), SHAPE),
        (dict(kc=fake((7, 16, 3, 128)), vc=fake((7, 16, 3, 128))), SHAPE), (dict(d=96), UNSUPPORTED), (dict(d=512), UNSUPPORTED),
        (dict(kv=0), SHAPE), (dict(t=MOST + 1), SHAPE),
        (dict(k=fake(s, addr=0x1008)), LAYOUT), (dict(k=fake(s, strides=(260, 128, 1))), LAYOUT), (dict(k=fake(s, strides=(512, 256, 2))), LAYOUT),
        (dict(kc=fake(c, strides=(2048, 256, 128, 1))), LAYOUT), (dict(kc=fake(c, strides=(0, 256, 128, 1))), LAYOUT),
        (dict(kc=kc, k=fake(s, addr=kc.data + 256)), LAYOUT), (dict(kc=kc, vc=fake(c, addr=kc.data)), LAYOUT),
        (dict(kc=kc, vc=fake(c, addr=kc.data + 256)), LAYOUT),
    ]:
        expect(store(lib, **kw), want)
    none = dict(k=fake((0, 2, 128), addr=0), v=fake((0, 2, 128), addr=0), slots=fake((0,), I64, addr=0))
    expect(store(lib, t=0, **none), 0)
    # the halves of one allocation [pages, 2, page, kv, d] pass its checks
    both = fake((14, 16, 2, 128))
    half = dict(strides=(2 * 16 * 256, 256, 128, 1))
    expect(store(lib, t=0, kc=fake(c, addr=both.data, **half), vc=fake(c, addr=both.data + 16 * 256 * 2, **half), **none), 0)


# ---------------------------------------------------------------------------
# attention


def prefill(lib, t=20, H=4, kv=2, d=128, dtype=BF16, o=None, **kw):
    a = dict(q=fake((t, H, d), dtype), k=fake((t, kv, d), dtype), v=fake((t, kv, d), dtype), cu=None, table=None, lens=None,
             out=fake((t, H, d), dtype))
    a.update(kw)
    return lib.gdn_attn_prefill(*[ref(a[n]) for n in ("q", "k", "v", "cu", "table", "lens", "out")], ref(o), None)


def paged(N=1, width=8, kv=2, d=128, pages=7, page=16, dtype=BF16, **kw):
    return {**dict(k=fake((pages, page, kv, d), dtype), v=fake((pages, page, kv, d), dtype), table=fake((N, width), I32), lens=fake((N,), I32)),
            **kw}


def test_prefill_refusals(lib):
    s, n = (20, 4, 128), (20, 2, 128)
    q, k = fake(s), fake(n)
    far = (1 << 24) + 8
    for kw, want in [
        *[({x: None}, NULL_ARG) for x in ("q", "k", "v", "out")],
        (dict(table=fake((1, 8), I32)), NULL_ARG), (dict(lens=fake((1,), I32)), NULL_ARG),
        (dict(dtype=I32), DTYPE), (dict(k=fake(n, F32)), DTYPE), (dict(v=fake(n, F32)), DTYPE), (dict(out=fake(s, F32)), DTYPE),
        (dict(d=96), UNSUPPORTED), (dict(d=32), UNSUPPORTED), (dict(out=fake((20, 4, 64))), SHAPE), (dict(out=fake((21, 4, 128))), SHAPE),
        (dict(out=fake((1, 20, 4, 128))), SHAPE), (dict(k=fake((19, 2, 128))), SHAPE), (dict(v=fake((20, 1, 128))), SHAPE),
        (dict(k=fake((20, 2, 64))), SHAPE), (dict(k=fake((1, 20, 2, 128)), v=fake((1, 20, 2, 128))), SHAPE),
        (dict(H=5), SHAPE), (dict(H=0, q=fake((20, 0, 128), addr=0), out=fake((20, 0, 128), addr=0)), SHAPE), (dict(H=65536, kv=1), UNSUPPORTED),
        (dict(cu=fake((4,), F32)), DTYPE), (dict(cu=fake((0,), I32, addr=0)), SHAPE),
        (dict(o=options(scale=float("nan"))), SHAPE), (dict(o=options(scale=float("inf"))), SHAPE), (dict(o=options(scale=2.0 ** 65)), SHAPE),
        (dict(o=options(window=-1)), SHAPE), (dict(o=options(sinks=-1)), SHAPE),
        (dict(q=fake(s, addr=0x1008)), LAYOUT), (dict(k=fake(n, strides=(260, 128, 1))), LAYOUT), (dict(v=fake(n, strides=(512, 256, 2))), LAYOUT),
        (dict(k=fake(n, strides=(far, 128, 1))), LAYOUT), (dict(v=fake(n, strides=(far, 128, 1))), LAYOUT),
        (dict(out=fake(s, strides=(512, 0, 1))), LAYOUT), (dict(q=q, out=fake(s, addr=q.data)), LAYOUT),
        (dict(k=k, out=fake(s, addr=k.data + 4096)), LAYOUT),
        # behind a cache
        (paged(N=2), SHAPE), (paged(N=2, cu=fake((4,), I32)), SHAPE), (paged(lens=fake((2,), I32)), SHAPE),
        (paged(lens=fake((1,), I64)), DTYPE), (paged(table=fake((1, 8), I64)), DTYPE), (paged(table=fake((1, 8), I32, strides=(8, 2))), LAYOUT),
        (paged(kv=3), SHAPE), (paged(d=64), SHAPE), (paged(width=1 << 28), SHAPE), (paged(v=fake((7, 16, 1, 128))), SHAPE),
        (paged(k=fake((7, 16, 2, 128), strides=(1 << 30, far, 128, 1))), LAYOUT), (paged(dtype=F32), DTYPE),
    ]:
        expect(prefill(lib, **kw), want)
    none = dict(q=fake((0, 4, 128), addr=0), out=fake((0, 4, 128), addr=0))
    expect(prefill(lib, t=0, k=fake((0, 2, 128), addr=0), v=fake((0, 2, 128), addr=0), **none), 0)
    expect(prefill(lib, t=0, **none, **paged()), 0)
    expect(prefill(lib, t=1000, H=1 << 12, kv=1, cu=fake((4097,), I32)), SHAPE)
    assert "pairs" in message()


def decode(lib, N=3, H=4, kv=2, d=128, dtype=BF16, o=None, ws=1 << 40, **kw):
    a = dict(q=fake((N, H, d), dtype), out=fake((N, H, d), dtype), **paged(N=N, kv=kv, d=d, dtype=dtype))
    a.update(kw)
    q, need = a["q"], ctypes.c_size_t(0)
    lib.gdn_attn_workspace_size(ref(q) if q is not None else ref(a["out"]), ctypes.byref(need))
    need = a.get("need", need.value)
    return lib.gdn_attn_decode(*[ref(a[n]) for n in ("q", "k", "v", "table", "lens", "out")], ref(o), ws, need, None)


def test_decode_refusals(lib):
    s, c = (3, 4, 128), (7, 16, 2, 128)
    q, k = fake(s), fake(c)
    for kw, want in [
        *[({x: None}, NULL_ARG) for x in ("q", "k", "v", "table", "lens", "out")],
        (dict(dtype=I32), DTYPE), (dict(k=fake(c, F32)), DTYPE), (dict(out=fake(s, F32)), DTYPE), (dict(lens=fake((3,), I64)), DTYPE),
        (dict(table=fake((3, 8), F32)), DTYPE), (dict(d=80), UNSUPPORTED), (dict(out=fake((3, 4, 64))), SHAPE),
        (dict(q=fake((1, 3, 4, 128)), out=fake((1, 3, 4, 128))), SHAPE), (dict(table=fake((2, 8), I32)), SHAPE), (dict(lens=fake((2,), I32)), SHAPE),
        (dict(v=fake((7, 8, 2, 128))), SHAPE), (dict(k=fake((7, 16, 2, 64)), v=fake((7, 16, 2, 64))), SHAPE), (dict(H=3), SHAPE),
        (dict(H=1 << 16, kv=1), UNSUPPORTED), (dict(N=(1 << 20) + 1), SHAPE), (dict(ws=None), WORKSPACE), (dict(ws=(1 << 40) + 64), WORKSPACE),
        (dict(need=100), WORKSPACE), (dict(o=options(scale=float("inf"))), SHAPE), (dict(o=options(window=-5)), SHAPE),
        (dict(o=options(sinks=-5)), SHAPE), (dict(q=fake(s, addr=0x1008)), LAYOUT), (dict(k=fake(c, strides=(4100, 256, 128, 1))), LAYOUT),
        (dict(k=fake(c, strides=(1 << 30, (1 << 24) + 8, 128, 1))), LAYOUT), (dict(out=fake(s, strides=(128, 128, 1))), LAYOUT),
        (dict(q=q, out=fake(s, addr=q.data)), LAYOUT), (dict(k=k, out=fake(s, addr=k.data + 256)), LAYOUT), (dict(k=k, ws=k.data), LAYOUT),
        (dict(lens=fake((3,), I32, strides=(2,))), LAYOUT), (dict(table=fake((3, 8), I32, addr=0)), NULL_ARG),
    ]:
        expect(decode(lib, **kw), want)
    expect(decode(lib, N=0, q=fake((0, 4, 128), addr=0), out=fake((0, 4, 128), addr=0), table=fake((0, 8), I32, addr=0),
                  lens=fake((0,), I32, addr=0)), 0)


def test_decode_workspace_follows_dtype_and_d_alone(lib):
    n = ctypes.c_size_t(0)
    for dtype in (BF16, F32):
        for d in (64, 128, 256):
            sizes = set()
            for N, H in ((1, 1), (300, 64), (1 << 20, 8), (0, 4)):
                q = fake((N, H, d), dtype)
                expect(lib.gdn_attn_workspace_size(ref(q), ctypes.byref(n)), 0)
                sizes.add(n.value)
            assert len(sizes) == 1 and 0 < n.value < 1 << 26 and n.value % 256 == 0
    for q, want in ((fake((3, 4, 96)), UNSUPPORTED), (fake((3, 128)), SHAPE), (fake((3, 4, 128), I32), DTYPE), (None, NULL_ARG)):
        expect(lib.gdn_attn_workspace_size(ref(q) if q else None, ctypes.byref(n)), want)
    q = fake((3, 4, 128))
    expect(lib.gdn_attn_workspace_size(ref(q), None), NULL_ARG)


# ---------------------------------------------------------------------------
# the header and the binding


def test_options_struct_matches_the_header(lib, tmp_path):
    src = tmp_path / "l.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "gdn.h"\nint main(void) {\n'
                   '  printf("%zu", sizeof(gdn_attn_options));\n' +
                   "".join(f'  printf(" %zu", offsetof(gdn_attn_options, {f}));\n' for f, _ in T.GdnAttnOptions._fields_) +
                   "  return 0;\n}\n")
    exe = tmp_path / "l"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", f"-I{ROOT}/include", str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(T.GdnAttnOptions)] + [getattr(T.GdnAttnOptions, f).offset for f, _ in T.GdnAttnOptions._fields_]
    o = T.gdn_attn_default_options()
    assert (o.scale, o.window, o.sinks) == (0.0, 0, 0)


def test_binding_refuses_cpu_tensors():
    import gated_deltanet_02_amd as G
    x, c, i, t = torch.randn(4, 2, 64), torch.randn(3, 16, 2, 64), torch.zeros(4, dtype=torch.int32), torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: G.gdn_cache_plan(i, 16, t, i, i[:1]), lambda: G.gdn_cache_release(i, i, 16, t, i, i[:1]),
                 lambda: G.gdn_cache_store(x, x, i.long(), c, c), lambda: G.gdn_attn_prefill(x, x, x), lambda: G.gdn_attn_decode(x, c, c, t, i)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
