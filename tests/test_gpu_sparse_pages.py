"""Attention over lists of large pages (nk_paged_sparse_attn): it takes every shape that the tensor-core decode takes, and
refuses the others before anything is launched."""
import numpy as np
import pytest
import torch

import quantized_paged_kv_cache_gb300 as nk
from quantized_paged_kv_cache_gb300 import workloads as wl

import _long_ref as ref
from _cases import build, compare

pytestmark = pytest.mark.gpu

# the most query heads of a kv-head at head dim 256, by page size (48 at every other size and head dim)
MOST = {112: 40, 128: 32, 144: 24, 160: 16, 176: 8, 192: 8}


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def case(D, P, G, lens, T=2, Hkv=1):
    w = wl.custom(f"d{D}_p{P}_g{G}", B=len(lens), T=T, Hq=G * Hkv, Hkv=Hkv, D=D, P=P, ctx_lens=lens, seed=29,
                  num_pages=sum(-(-L // P) for L in lens) + 1)
    c = build(w, fill=0xFF, oracle_pool=False)
    c.status = i32([0])
    return c


def run_and_check(c, k, **kw):
    """Random lists: pages in any order, entries that name none behind and between."""
    w = c.w
    rng = np.random.RandomState(k)
    lists = np.full((w.B, w.T, w.Hkv, k), -1)
    for b in range(w.B):
        for t in range(w.T):
            for h in range(w.Hkv):
                seen = (w.ctx_lens[b] - w.T + t) // w.P + 1
                pick = rng.permutation(seen)[:rng.randint(1, k + 1)]
                lists[b, t, h, :len(pick)] = pick
    out = nk.paged_sparse_attn(c.pool, c.q, c.bt, c.ctx, i32(lists), w.sm_scale, w.max_ctx, status=c.status, **kw)
    assert int(c.status.item()) == 0
    compare(out, ref.sparse(c.pool.storage, w.num_pages, w.Hkv, w.P, w.D, c.bt_cpu.numpy(), w.ctx_lens, lists, c.q, w.sm_scale), w.name)


@pytest.mark.parametrize("D,P,G", [(256, P, G) for P, G in MOST.items()] + [(256, 192, 1), (128, 256, 41), (128, 256, 48), (64, 256, 48),
                                   (256, 96, 48)])
def test_large_pages(D, P, G):
    run_and_check(case(D, P, G, [9 * P + 5, 3 * P - 1]), 5)


@pytest.mark.parametrize("D,P,G", [(256, 192, 6), (128, 256, 42)])
def test_many_large_pages_of_one_block(D, P, G):
    """More pages than a block keeps the numbers of, several sequences in its range."""
    run_and_check(case(D, P, G, [65, 40 * P, 11 * P + 7, 30 * P + 1] + [17 * P + i for i in range(28)], T=1), 24, num_ctas=1)


def test_what_fits_is_what_the_tensor_core_decode_takes():
    one, none = i32([1]), i32([[0]])
    for D in (64, 128, 256):
        for P in range(16, 257, 16):
            pool = nk.KVPool(torch.zeros(nk.kv_pool_bytes(1, P, 1, D), dtype=torch.uint8, device="cuda"), 1, P, 1, D)
            for G in range(1, 49):
                q = torch.zeros((1, 1, G, D), dtype=torch.bfloat16, device="cuda")
                fits = G <= (48 if D < 256 or P <= 96 else MOST.get(P, 0))
                try:
                    nk.paged_sparse_attn(pool, q, none, one, none.view(1, 1, 1, 1), 0.1, 1)
                    assert fits, (D, P, G)
                except nk.NKError as e:
                    assert not fits and e.code == 3, (D, P, G, e)
    torch.cuda.synchronize()
