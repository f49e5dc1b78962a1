"""The mma.sync decode on page sizes whose ring is no whole number of the teams' rounds (the waits then ask whether a page
was issued), or was cut to one, over contexts that go around it many times; against the plain 64-bit form, run to run the
same, and with pages that are never loaded."""
import pytest
import torch

import quantized_paged_kv_cache_gb300 as nk
from quantized_paged_kv_cache_gb300 import workloads as wl

import _ref
from _cases import build, compare

pytestmark = pytest.mark.gpu

SHAPES = [
    # Hq, Hkv, D, P, T
    (6, 1, 256, 80, 1),
    (12, 2, 256, 112, 1),
    (12, 1, 256, 48, 1),
    (24, 1, 256, 48, 1),
    (8, 1, 128, 112, 1),
    (24, 1, 128, 96, 1),
    (16, 2, 128, 16, 2),
    (20, 1, 128, 16, 1),
    (20, 1, 256, 16, 1),
    (40, 1, 64, 64, 1),
    (8, 8, 64, 48, 1),
]


@pytest.mark.parametrize("Hq,Hkv,D,P,T", SHAPES)
def test_many_rounds_of_the_ring(Hq, Hkv, D, P, T):
    lens = [9001, 700]
    w = wl.custom(f"ring{D}_{P}", B=2, T=T, Hq=Hq, Hkv=Hkv, D=D, P=P, ctx_lens=lens, seed=98,
                  num_pages=sum((L + P - 1) // P for L in lens) + 2)
    c = build(w, fill=0xFF, oracle_pool=False)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def reference(window, sinks):
        return _ref.attention(c.pool.storage, w.num_pages, Hkv, P, D, c.bt, lens, [T] * 2, c.q, w.sm_scale, window,
                              sinks).cpu().numpy()

    args = (c.pool, c.q, c.bt, c.ctx, w.sm_scale, w.max_ctx)
    for what, call, ref in (
            ("whole", lambda n: nk.paged_decode_attn(*args, num_ctas=n, status=status), reference(0, 0)),
            ("window", lambda n: nk.paged_window_attn(*args, 6000, sinks=20, num_ctas=n, status=status), reference(6000, 20))):
        for n in (1, 3, 0):
            out = call(n)
            compare(out, ref, f"{w.name} {what} ctas={n}")
            for _ in range(5):
                assert torch.equal(out, call(n)), f"{what} ctas={n}: run-to-run results differ"
    assert int(status.item()) == 0


@pytest.mark.parametrize("Hq,Hkv,D,P,T", SHAPES[:3])
@pytest.mark.parametrize("withheld", [0, 2, 9])
def test_pages_that_are_never_loaded_time_out(Hq, Hkv, D, P, T, withheld):
    w = wl.custom(f"ringstall{D}_{P}", B=1, T=T, Hq=Hq, Hkv=Hkv, D=D, P=P, ctx_lens=[4000], seed=99,
                  num_pages=4000 // P + 2)
    c = build(w, oracle_pool=False)
    run = lambda s: nk.paged_decode_attn(c.pool, c.q, c.bt, c.ctx, w.sm_scale, w.max_ctx, num_ctas=2, status=s)  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = run(status)
    torch.cuda.synchronize()
    try:
        nk.test_inject_copy_stall(withheld, 1 << 20)
        run(status)
        torch.cuda.synchronize()
    finally:
        nk.test_inject_copy_stall(-1)
    assert int(status.item()) & nk.NK_DEVFLAG_TIMEOUT
    status.zero_()
    assert torch.equal(run(status), want) and int(status.item()) == 0
