"""The operators over long caches at byte offsets past 32 bits: the same pages,
bounds and rows at the end of a large buffer give the same bits."""
import numpy as np
import pytest
import torch

import quantized_paged_kv_cache_gb300 as nk

from test_gpu_sparse import i32, make, made_bounds
from test_gpu_verify import case, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 4, 16])  # (16: 96 rows of a kv-head, the tcgen05 kernel of the weights)
def test_pages_past_4_gib(T):
    c = make(("far", 2, T, 24, 4, 256, 64, [1500, 333]))
    w = c.w
    page = c.pool.storage.numel() // w.num_pages
    total = (1 << 32) // page + 2 * w.num_pages
    far = total - w.num_pages
    assert far * page > 1 << 32
    storage = torch.empty(total * page, dtype=torch.uint8, device="cuda")
    storage[far * page:] = c.pool.storage
    pool = nk.KVPool(storage, total, w.P, w.Hkv, w.D)
    bt = torch.where(c.bt >= 0, c.bt + far, c.bt)
    start, cu = i32([0] * w.B), i32(np.cumsum([0] + list(w.ctx_lens)))
    near_b, far_b = made_bounds(c), nk.PageBounds.empty(pool)
    nk.page_bounds(pool, far_b, bt, start, cu, status=c.status)
    assert torch.equal(far_b.codes()[far:], near_b.codes()) and torch.equal(far_b.scales()[far:], near_b.scales())
    near_p = nk.page_select(near_b, c.q, c.bt, c.ctx, w.P, w.max_ctx, 4, status=c.status)
    far_p = nk.page_select(far_b, c.q, bt, c.ctx, w.P, w.max_ctx, 4, status=c.status)
    assert torch.equal(far_p, near_p)
    near_o = nk.paged_sparse_attn(c.pool, c.q, c.bt, c.ctx, near_p, w.sm_scale, w.max_ctx, status=c.status)
    assert torch.equal(nk.paged_sparse_attn(pool, c.q, bt, c.ctx, near_p, w.sm_scale, w.max_ctx, status=c.status), near_o)
    near_w, far_w = (torch.zeros((n, w.Hkv), device="cuda") for n in (w.num_pages, total))
    nk.page_weights(c.pool, c.q, c.bt, c.ctx, w.sm_scale, w.max_ctx, near_w, status=c.status)
    nk.page_weights(pool, c.q, bt, c.ctx, w.sm_scale, w.max_ctx, far_w, status=c.status)
    assert torch.equal(far_w[far:], near_w) and not far_w[:far].any()
    assert int(c.status.item()) == 0


def test_bounds_past_4_gib():
    c = make(("far", 2, 2, 24, 4, 256, 64, [1500, 333]))
    w, b = c.w, made_bounds(c)
    total = (1 << 32) // (w.Hkv * 2 * w.D) + 2 * w.num_pages
    far = total - w.num_pages
    big = nk.PageBounds(torch.zeros(nk.page_bounds_bytes(total, w.Hkv, w.D), dtype=torch.uint8, device="cuda"), total, w.Hkv, w.D)
    big.codes()[far:] = b.codes()
    big.scales()[far:] = b.scales()
    bt = torch.where(c.bt >= 0, c.bt + far, c.bt)
    want = nk.page_select(b, c.q, c.bt, c.ctx, w.P, w.max_ctx, 5, status=c.status)
    assert torch.equal(nk.page_select(big, c.q, bt, c.ctx, w.P, w.max_ctx, 5, status=c.status), want)
    values = big.values()
    assert torch.equal(values[far:], b.values()) and not values[:3].any() and not values[far - 3:far].any()
    assert int(c.status.item()) == 0


def test_probabilities_past_4_gib():
    p, q, d, u = case(2, 4, 999, 21)
    row = (1 << 28) + 8  # 1 GiB and 32 bytes
    big = torch.empty(8 * row, device="cuda")
    ps, qs = big.as_strided(p.shape, (4 * row, row, 1)), big.as_strided(q.shape, (3 * row, row, 1), 2000)
    ps.copy_(p)
    qs.copy_(q)
    check(ps, qs, d, u)
