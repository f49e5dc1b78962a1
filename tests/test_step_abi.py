"""Host-side refusals of the step operators, before anything is launched (CPU only)."""
import ctypes

import pytest

import quantized_paged_kv_cache_gb300 as nk
from quantized_paged_kv_cache_gb300 import _lib

FAKE = 1 << 20  # never dereferenced: every call below fails host validation first


def pool(num_pages=16, P=16, H=1, D=64, base=FAKE):
    return _lib.nk_kv_pool(base, num_pages, P, H, D)


def test_step_tables_refusals():
    def call(P=16, pages=8, start=FAKE, new=FAKE + 64, B=2, free=FAKE, n=4, table=FAKE, width=4, cu=FAKE, ctx=FAKE + 128,
             slots=FAKE, pos=FAKE, rows=8):
        return nk.lib().nk_step_tables(P, pages, start, new, B, free, n, table, width, cu, ctx, slots, pos, rows, None,
                                       None, None)

    assert call(B=0, cu=None) == 1  # (a step of no sequences still writes cu_new[0])
    assert call(P=0) == 2 and call(pages=0) == 2 and call(B=-1) == 2 and call(n=-1) == 2 and call(width=0) == 2
    assert call(rows=-1) == 2
    assert call(B=1025) == 3
    for name in ("start", "new", "free", "table", "cu", "ctx", "slots"):
        assert call(**{name: None}) == 1, name
    assert call(ctx=FAKE) == 2 and call(ctx=FAKE + 64) == 2  # the lengths, overwritten while they are read


def test_mrope_refusals():
    def call(q=FAKE, k=FAKE, qo=FAKE * 2, ko=FAKE * 2, qs=512, ks=128, qos=512, kos=128, rows=2, Hq=4, Hkv=1, D=128,
             pos=FAKE, ps=2, inv=(1.0,) * 64, sections=(32, 16, 16), axes=None, inter=0):
        axes = len(sections) if axes is None else axes
        fr = (ctypes.c_double * len(inv))(*inv) if inv is not None else None
        se = (ctypes.c_int32 * len(sections))(*sections)
        return nk.lib().nk_mrope(q, k, qo, ko, qs, ks, qos, kos, rows, Hq, Hkv, D, pos, ps, fr, se, axes, inter, None,
                                 None)

    assert call(rows=0) == 0
    assert call(rows=-1) == 2 and call(Hq=0, Hkv=0) == 2 and call(D=260) == 2 and call(D=100) == 2 and call(D=8) == 2
    assert call(axes=0) == 2 and call(axes=5, sections=(8,) * 5) == 2
    assert call(sections=(32, -16, 16)) == 2 and call(sections=(30, 16, 16)) == 2 and call(sections=(0, 0, 0)) == 2
    assert call(sections=(32, 32, 16)) == 2  # more than half a head
    assert call(inv=None) == 1 and call(pos=None) == 1 and call(q=None) == 1 and call(ko=None) == 1
    assert call(inv=(float("inf"),) * 64) == 2
    assert call(qs=500) == 2 and call(qs=516) == 2 and call(kos=64) == 2 and call(ps=1) == 2
    assert call(q=FAKE + 2) == 2 and call(ko=FAKE + 8) == 2
    assert call(qo=FAKE, qos=1024) == 2  # in place with another stride


def test_window_refusals():
    def call(p=pool(), q=FAKE, T=1, Hq=2, B=1, max_ctx=64, window=8, sinks=0, n=0, wsb=1 << 30, out=FAKE, scale=0.1):
        return nk.lib().nk_paged_window_attn(ctypes.byref(p) if p is not None else None, q, FAKE, 4, FAKE, B, T, Hq,
                                             scale, max_ctx, window, sinks, n, FAKE, wsb, out, None, None)

    assert call(window=0) == 2 and call(sinks=-1) == 2
    assert call(p=None) == 1 and call(q=None) == 1 and call(out=None) == 1
    assert call(T=0) == 2 and call(T=17) == 2 and call(Hq=3, p=pool(H=2)) == 2 and call(max_ctx=65) == 2
    assert call(scale=float("nan")) == 2 and call(q=FAKE + 2) == 2
    assert call(wsb=16) == 4
    assert call(B=1025) == 3 and call(Hq=49) == 3  # more than 48 rows of one kv-head
    assert call(B=0) == 0
    # a split that gives one CTA more than 262,144 keys: refused when the window is that long, not for a short one
    big = pool(num_pages=1 << 14, P=64, H=4, D=256)

    def far(window, wsb):
        return nk.lib().nk_paged_window_attn(ctypes.byref(big), FAKE, FAKE, 1 << 14, FAKE, 1, 1, 24, 0.1, 1 << 20, window,
                                             0, 4, FAKE, wsb, FAKE, None, None)

    assert far(1 << 19, 1 << 40) == 3
    assert far(1 << 12, 16) == 4  # past that check: the workspace is refused next


def test_binding_refusals():
    import torch

    z = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        nk.step_tables(16, 8, z, z, z, z.view(4, 1), z, z, z.long())  # host tensors
    x = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        nk.mrope(x, x[:, :1], torch.zeros(3, 2, dtype=torch.int32), torch.ones(64, dtype=torch.float64), (32, 16, 16))
    with pytest.raises(ValueError):
        nk.mrope(x, x[:1, :1], torch.zeros(3, 2, dtype=torch.int32), torch.ones(64, dtype=torch.float64), (32, 16, 16))


def test_chunk_refusals():
    need = nk.chunk_workspace_bytes(64, 4)
    assert need >= 4 * 2 * 128 * 65 * 4 and nk.chunk_workspace_bytes(96, 4) == 0

    def call(p=pool(), q=FAKE, cu=FAKE, B=1, total=5, Hq=2, max_ctx=64, window=0, sinks=0, n=4, ws=FAKE, wsb=need, out=FAKE * 2,
             scale=0.1, pages=4):
        return nk.lib().nk_paged_chunk_attn(ctypes.byref(p) if p is not None else None, q, cu, FAKE, pages, FAKE, B, total,
                                            Hq, scale, max_ctx, window, sinks, n, ws, wsb, out, None, None)

    assert call(p=None) == 1 and call(q=None) == 1 and call(cu=None) == 1 and call(out=None) == 1
    assert call(B=-1) == 2 and call(total=-1) == 2 and call(window=-1) == 2 and call(sinks=-1) == 2
    assert call(Hq=3, p=pool(H=2)) == 2 and call(Hq=0) == 2 and call(max_ctx=65) == 2 and call(max_ctx=0) == 2
    assert call(pages=0) == 2 and call(scale=float("inf")) == 2 and call(q=FAKE + 8) == 2 and call(p=pool(P=24)) == 2
    assert call(total=1 << 30, Hq=4) == 2 and call(n=1 << 21) == 2
    assert call(out=FAKE) == 2  # over the queries
    assert call(B=1025) == 3
    assert call(ws=None) == 4 and call(wsb=need - 1) == 4 and call(ws=FAKE + 4) == 4
    assert call(B=0) == 0 and call(total=0) == 0
