"""Windowed chunks over pages of fewer than 64 keys: only the pages that hold a key some token of the chunk sees are looked
up and read, so the pages between the sinks and the window may have been given back (their entries -1, or handed to others)."""
import pytest
import torch

import quantized_paged_kv_cache_gb300 as nk

from test_gpu_chunk import Chunk, check

pytestmark = pytest.mark.gpu

SHAPES = [
    # query tokens, contexts, Hq, Hkv, D, P
    ([70, 1, 5], [2000, 1111, 700], 24, 4, 256, 16),
    ([70, 1, 300], [2000, 1111, 700], 16, 2, 128, 16),
    ([33, 1, 64], [1999, 1024, 129], 8, 2, 128, 32),
    ([100, 1], [1500, 777], 10, 2, 64, 48),
    ([10, 1], [1500, 777], 10, 2, 64, 80),
    ([70, 1], [2000, 1111], 6, 2, 128, 64),
]


@pytest.mark.parametrize("window,sinks", [(200, 70), (1, 0), (33, 1), (65, 17), (150, 0), (10, 130)])
@pytest.mark.parametrize("shape", SHAPES, ids=[f"d{s[4]}_p{s[5]}" for s in SHAPES])
def test_pages_given_back_are_not_read(shape, window, sinks):
    qlens, ctx, Hq, Hkv, D, P = shape
    k = Chunk("freed", qlens, ctx, Hq, Hkv, D, P, seed=83)
    want = k.run(window, sinks)
    check(want, k.ref(window, sinks), "all pages there")
    bt, other = k.c.bt.clone(), k.c.bt.clone()
    used = {int(x) for b, L in enumerate(ctx) for x in k.c.bt[b, :-(-L // P)]}
    spare = min(set(range(k.w.num_pages)) - used)  # no sequence's page here: full of another's (non-finite) rows
    k.c.pool.storage.view(k.w.num_pages, -1)[spare] = 0xFF
    freed = 0
    for b, (L, T) in enumerate(zip(ctx, qlens)):
        first, lead = max(0, L - T - window + 1) // P, -(-sinks // P)
        if first > lead:
            bt[b, lead:first] = -1
            other[b, lead:first] = spare
            freed += first - lead
        bt[b, -(-L // P):] = 1 << 30
    assert freed > 0
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for table in (bt, other):
        for n in (0, 1, 5):
            out = k.run(window, sinks, bt=table, status=status, num_ctas=n)
            torch.cuda.synchronize()
            assert int(status.item()) == 0
            if n == 0:
                assert torch.equal(out, want)
            else:
                check(out, k.ref(window, sinks), f"ctas={n}")
