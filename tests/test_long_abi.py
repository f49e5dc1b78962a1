"""Host-side refusals of the operators over long caches and of draft
verification, before anything is launched (CPU only)."""
import ctypes

import pytest

import quantized_paged_kv_cache_gb300 as nk
from quantized_paged_kv_cache_gb300 import _lib

FAKE = 1 << 20  # never dereferenced: every call below fails host validation first


def pool(num_pages=16, P=16, H=1, D=64, base=FAKE):
    return _lib.nk_kv_pool(base, num_pages, P, H, D)


def ref(p):
    return ctypes.byref(p) if p is not None else None


def test_sizes():
    assert nk.page_bounds_bytes(10, 4, 256) == 10 * 4 * (2 * 256 + 4) and nk.page_bounds_bytes(10, 4, 96) == 0
    assert nk.page_bounds_bytes(1 << 24, 8, 256) == (1 << 27) * 516
    assert nk.page_select_workspace_bytes(8, 4, 24, 4, 256, 64, 65536) == 0  # in one launch
    assert nk.page_select_workspace_bytes(8, 16, 24, 4, 256, 64, 65536) == 8 * 16 * 4 * 1024 * 8  # 96 rows of a kv-head
    assert nk.page_select_workspace_bytes(1, 1, 4, 2, 64, 16, 20000 * 16) == 2 * 20000 * 8  # more pages than stay on chip
    assert nk.page_select_workspace_bytes(0, 1, 1, 1, 64, 16, 17) == 0
    one = nk.page_weights_workspace_bytes(1, 1, 6, 1, 16, 100)
    assert one == (7 + 7 + 1) * 8 * 4  # seven pages, as many CTAs, one unit, six rows in a tile of eight
    assert nk.page_weights_workspace_bytes(1, 17, 6, 1, 16, 100) == 0


def test_bounds_refusals():
    def call(p=pool(), bounds=FAKE, bt=FAKE, width=4, start=FAKE, cu=FAKE, B=1):
        return nk.lib().nk_page_bounds(ref(p), bounds, bt, width, start, cu, B, None, None)

    assert call(p=None) == 1 and call(p=pool(base=None)) == 1
    for name in ("bounds", "bt", "start", "cu"):
        assert call(**{name: None}) == 1, name
    assert call(p=pool(P=24)) == 2 and call(p=pool(D=96)) == 2 and call(width=0) == 2 and call(B=-1) == 2 and call(bounds=FAKE + 8) == 2
    assert call(B=1025) == 3 and call(B=0) == 0


def test_bounds_values_refusals():
    def call(bounds=FAKE, pages=2, H=1, D=64, out=FAKE):
        return nk.lib().nk_page_bounds_values(bounds, pages, H, D, out, None)

    assert call(bounds=None) == 1 and call(out=None) == 1
    assert call(pages=0) == 2 and call(H=0) == 2 and call(D=96) == 2 and call(bounds=FAKE + 8) == 2 and call(out=FAKE + 4) == 2


def test_select_refusals():
    def call(bounds=FAKE, pages=16, P=16, Hkv=2, D=64, q=FAKE, bt=FAKE, width=8, ctx=FAKE, B=2, T=2, Hq=4, max_ctx=128, k=4, sinks=1,
             recent=1, ws=None, wsb=0, out=FAKE):
        return nk.lib().nk_page_select(bounds, pages, P, Hkv, D, q, bt, width, ctx, B, T, Hq, max_ctx, k, sinks, recent, ws, wsb, out, None, None)

    for name in ("bounds", "q", "bt", "ctx", "out"):
        assert call(**{name: None}) == 1, name
    for bad in (dict(pages=0), dict(P=0), dict(Hkv=0), dict(D=96), dict(B=-1), dict(T=0), dict(T=17), dict(Hq=3), dict(k=0), dict(sinks=-1),
                dict(recent=0), dict(sinks=4), dict(sinks=2**31 - 1), dict(width=0), dict(max_ctx=129), dict(max_ctx=1), dict(bounds=FAKE + 4),
                dict(q=FAKE + 2)):
        assert call(**bad) == 2, bad
    assert call(Hq=2 * 49) == 3 and call(B=40000) == 3 and call(B=0) == 0
    many = dict(T=16, Hq=2 * 5, wsb=2 * 16 * 2 * 8 * 8, ws=FAKE)  # 80 rows: two launches, which need a workspace
    assert call(**many | dict(ws=None)) == 4 and call(**many | dict(wsb=4095)) == 4 and call(**many | dict(ws=FAKE + 8)) == 4


def test_sparse_refusals():
    def call(p=pool(), q=FAKE, lists=FAKE, k=4, T=1, Hq=2, B=1, max_ctx=64, n=0, ws=FAKE, wsb=1 << 30, out=FAKE, scale=0.1):
        return nk.lib().nk_paged_sparse_attn(ref(p), q, FAKE, 4, FAKE, lists, k, B, T, Hq, scale, max_ctx, n, ws, wsb, out, None, None)

    assert call(p=None) == 1 and call(q=None) == 1 and call(out=None) == 1 and call(lists=None) == 1
    assert call(k=0) == 2 and call(T=0) == 2 and call(T=17) == 2 and call(Hq=3, p=pool(H=2)) == 2 and call(max_ctx=65) == 2
    assert call(scale=float("nan")) == 2 and call(q=FAKE + 2) == 2
    assert call(ws=None) == 4 and call(wsb=16) == 4 and call(ws=FAKE + 4) == 4
    assert call(Hq=49) == 3 and call(B=65, T=16, max_ctx=64) == 3 and call(B=0) == 0
    big = pool(num_pages=1 << 16, P=64, H=1, D=64)
    assert nk.lib().nk_paged_sparse_attn(ref(big), FAKE, FAKE, 1 << 14, FAKE, FAKE, 1 << 13, 1, 1, 2, 0.1, 1 << 20, 1, FAKE, 1 << 40, FAKE, None,
                                         None) == 3  # 8,192 pages of 64 keys in one CTA


def test_weights_refusals():
    need = nk.page_weights_workspace_bytes(1, 1, 2, 1, 16, 64)

    def call(p=pool(), q=FAKE, bt=FAKE, ctx=FAKE, B=1, T=1, Hq=2, scale=0.1, max_ctx=64, ws=FAKE, wsb=need, out=FAKE):
        return nk.lib().nk_page_weights(ref(p), q, bt, 4, ctx, B, T, Hq, scale, max_ctx, None, None, ws, wsb, out, None, None)

    assert call(p=None) == 1 and call(q=None) == 1 and call(bt=None) == 1 and call(ctx=None) == 1 and call(out=None) == 1
    assert call(T=0) == 2 and call(T=17) == 2 and call(Hq=3, p=pool(H=2)) == 2 and call(max_ctx=65) == 2 and call(max_ctx=0) == 2
    assert call(scale=float("inf")) == 2 and call(q=FAKE + 8) == 2 and call(B=-1) == 2
    assert call(ws=None) == 4 and call(wsb=need - 1) == 4 and call(ws=FAKE + 8) == 4
    assert call(B=1025) == 3 and call(Hq=49) == 3 and call(B=0) == 0


def test_evict_refusals():
    def call(P=16, pages=8, Hkv=1, w=FAKE, bt=FAKE, out=FAKE, width=4, ctx=FAKE, B=1, keep=3, sinks=1, recent=1, new=FAKE * 2, freed=FAKE,
             most=4, count=FAKE):
        return nk.lib().nk_evict_pages(P, pages, Hkv, w, bt, out, width, ctx, B, keep, sinks, recent, new, freed, most, count, None, None)

    for name in ("w", "bt", "out", "ctx", "new", "freed", "count"):
        assert call(**{name: None}) == 1, name
    for bad in (dict(P=0), dict(pages=0), dict(Hkv=0), dict(B=-1), dict(width=0), dict(most=-1), dict(sinks=-1), dict(recent=0), dict(keep=1),
                dict(sinks=2**31 - 1), dict(new=FAKE)):
        assert call(**bad) == 2, bad
    assert call(B=1025) == 3 and call(width=16385) == 3 and call(B=0, count=None) == 1


def test_verify_refusals():
    def call(p=FAKE, ps=100, q=FAKE, qs=100, d=FAKE, n=None, u=FAKE, B=2, T=3, V=100, ctx=FAKE, tokens=FAKE * 2, acc=FAKE * 3, nxt=FAKE):
        return nk.lib().nk_verify_drafts(p, ps, q, qs, d, n, u, B, T, V, ctx, tokens, acc, nxt, None, None)

    for name in ("p", "d", "u", "tokens", "acc", "ctx"):
        assert call(**{name: None}) == 1, name
    assert call(T=0) == 2 and call(T=17) == 2 and call(V=0) == 2 and call(B=-1) == 2 and call(ps=99) == 2 and call(qs=99) == 2
    assert call(tokens=FAKE) == 2 and call(n=FAKE * 3) == 2  # results over what other blocks read
    assert call(B=65536) == 3 and call(V=(1 << 30) + 1, ps=1 << 31, qs=1 << 31) == 3 and call(B=0) == 0


def test_binding_refusals():
    import torch

    i = torch.zeros(4, dtype=torch.int32)
    f = torch.zeros(1, 1, 8)
    p = nk.KVPool(torch.zeros(4, dtype=torch.uint8), 1, 16, 1, 64)
    b = nk.PageBounds(torch.zeros(1000, dtype=torch.uint8), 1, 1, 64)
    q = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: nk.page_bounds(p, b, i.view(1, 4), i[:1], i[:2]), lambda: nk.page_select(b, q, i.view(1, 4), i[:1], 16, 16, 1),
                 lambda: nk.paged_sparse_attn(p, q, i.view(1, 4), i[:1], i.view(1, 1, 1, 4), 0.1, 16),
                 lambda: nk.page_weights(p, q, i.view(1, 4), i[:1], 0.1, 16, f[0]),
                 lambda: nk.evict_pages(16, f[0], i.view(1, 4), i[:1], 2, i[1:2], i, i[:1]),
                 lambda: nk.verify_drafts(f, None, i[:0], f[0, :, :1])):
        with pytest.raises(ValueError, match="CUDA"):  # host tensors
            call()
    with pytest.raises(ValueError, match="target"):
        nk.verify_drafts(f[0], None, i[:0], f[0, :, :1])
    with pytest.raises(ValueError, match="distance"):
        nk._vocab_stride(torch.zeros(3, 2, 8).transpose(0, 1), "target")
    assert nk._vocab_stride(torch.zeros(2, 3, 10)[..., :8], "target") == 10 and nk._vocab_stride(torch.zeros(2, 0, 8), "draft") >= 8
