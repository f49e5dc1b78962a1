"""Failure detection of the bounded waits in the kernels over long caches (GPU),
without a fault: some copies are simply never issued (nk_test_inject_copy_stall).
The call reports NK_DEVFLAG_TIMEOUT, returns within a fraction of a second, and the
next, normal call gives what the one before gave."""
import time

import numpy as np
import pytest
import torch

import quantized_paged_kv_cache_gb300 as nk
from quantized_paged_kv_cache_gb300 import workloads as wl

from _cases import build

pytestmark = pytest.mark.gpu

WAIT = 1 << 20  # cycles (~0.5 ms)


@pytest.fixture(autouse=True)
def no_injection_left():
    yield
    nk.test_inject_copy_stall(-1)


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("what,T", [("sparse", 2), ("bounds", 1), ("weights", 1), ("weights", 6), ("weights", 16)])
@pytest.mark.parametrize("withheld", [0, 1, 3])
def test_withheld_copies_time_out_and_the_device_recovers(what, T, withheld):
    lens = [40000, 30011]
    w = wl.custom(f"stall_{what}", B=2, T=T, Hq=8, Hkv=2, D=128, P=64, ctx_lens=lens, seed=57, num_pages=sum(-(-L // 64) for L in lens) + 1)
    c = build(w, oracle_pool=False)
    status = i32([0])
    if what == "sparse":
        lists = i32(np.broadcast_to(np.arange(40), (2, T, 2, 40)).copy())
        call = lambda: nk.paged_sparse_attn(c.pool, c.q, c.bt, c.ctx, lists, w.sm_scale, w.max_ctx, num_ctas=8, status=status)  # noqa: E731
    elif what == "weights":
        call = lambda: nk.page_weights(c.pool, c.q, c.bt, c.ctx, w.sm_scale, w.max_ctx,  # noqa: E731
                                       torch.zeros((w.num_pages, 2), device="cuda"), status=status)
    else:
        def call():
            b = nk.PageBounds.empty(c.pool)
            nk.page_bounds(c.pool, b, c.bt, i32([0, 0]), i32([0, lens[0], sum(lens)]), status=status)
            return b.storage
    want = call()
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    nk.test_inject_copy_stall(withheld, WAIT)
    t0 = time.perf_counter()
    call()
    torch.cuda.synchronize()
    elapsed = time.perf_counter() - t0
    nk.test_inject_copy_stall(-1)
    assert int(status.item()) & nk.NK_DEVFLAG_TIMEOUT
    assert elapsed < 1.0, f"the call took {elapsed:.3f} s"
    status.zero_()
    assert torch.equal(call(), want)
    assert int(status.item()) == 0
