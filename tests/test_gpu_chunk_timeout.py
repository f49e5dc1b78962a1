"""The ragged chunk attention's bounded waits where a CTA goes through many short segments: what its warps hand each other
about the segments lies in a ring of 16 slots, and a wait that runs out in an early one must not let the warp that fills the
ring run past those that read it. No GPU fault is involved: blocks are never handed over (nk_test_inject_copy_stall)."""
import time

import pytest
import torch

import quantized_paged_kv_cache_gb300 as nk

from test_gpu_chunk import Chunk, check

pytestmark = pytest.mark.gpu

WAIT = 1 << 20  # cycles (~0.5 ms)


@pytest.fixture(autouse=True)
def no_injection_left():
    yield
    nk.test_inject_copy_stall(-1)


@pytest.mark.parametrize("withheld", [0, 1, 5, 40])
@pytest.mark.parametrize("ctas", [1, 3])
def test_many_short_segments_after_a_wait_has_run_out(withheld, ctas):
    # 200 sequences of one token and one 64-key block, two kv-heads: 400 segments of one block (134 and more a CTA)
    ctx = [1 + 7 * b % 64 for b in range(200)]
    k = Chunk("segments", [1] * 200, ctx, 4, 2, 64, 16, seed=81)
    ref = k.ref()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    nk.test_inject_copy_stall(withheld, WAIT)
    t0 = time.perf_counter()
    k.run(num_ctas=ctas, status=status)
    torch.cuda.synchronize()
    elapsed = time.perf_counter() - t0
    nk.test_inject_copy_stall(-1)
    assert int(status.item()) & nk.NK_DEVFLAG_TIMEOUT
    assert elapsed < 1.0, f"the call took {elapsed:.3f} s"
    status.zero_()
    check(k.run(num_ctas=ctas, status=status), ref, "the call after it")
    assert int(status.item()) == 0
