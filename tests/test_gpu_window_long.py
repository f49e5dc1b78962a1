"""Windows of tens of thousands of keys run by one CTA (nk_paged_window_attn), against the plain 64-bit form: the tcgen05
decode's folding instance (more than 512 pages of one kv-head), page numbers past those it keeps in shared memory (512, and
1,024 on mma.sync), with the gap behind the sinks given back. The tolerance is the decode kernels' (4e-3, relative 1e-3 of
the rounded reference)."""
import pytest
import torch

import quantized_paged_kv_cache_gb300 as nk
from quantized_paged_kv_cache_gb300 import workloads as wl

from _cases import build, compare
from test_gpu_window import call, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,P,Hq,Hkv,T,ctx,window,sinks", [
    (256, 64, 6, 1, 2, [45003, 1000], 40000, 70),     # tcgen05: 627 pages, folded
    (256, 64, 6, 1, 4, [45003, 1000], 40000, 70),
    (256, 64, 6, 1, 5, [1000, 45003], 40001, 0),
    (128, 16, 8, 1, 1, [24011, 300], 20000, 70),      # mma.sync: 1,255 pages
    (256, 16, 6, 1, 1, [300, 24011], 20001, 5),
    (64, 48, 4, 1, 3, [61000], 56000, 130),
])
def test_a_long_window_in_one_cta(D, P, Hq, Hkv, T, ctx, window, sinks):
    w = wl.custom(f"longwin{D}_{P}_{T}", B=len(ctx), T=T, Hq=Hq, Hkv=Hkv, D=D, P=P, ctx_lens=ctx, seed=97,
                  num_pages=sum((L + P - 1) // P for L in ctx) + 2)
    c = build(w, fill=0xFF, oracle_pool=False)
    ref = reference(c, window, sinks)
    bt = c.bt.clone()
    for b, L in enumerate(ctx):
        first, lead = max(0, L - T - window + 1) // P, -(-sinks // P)
        if first > lead:
            bt[b, lead:first] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for n in (1, 2, 0):
        compare(call(c, window, sinks, bt=bt, num_ctas=n, status=status), ref, f"{w.name}/ctas={n}")
    assert int(status.item()) == 0
