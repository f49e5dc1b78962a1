"""Keys that lie in a page with the window's (or the sinks') but that no column sees: their K and V, of any size or not
finite, leave no trace in nk_paged_window_attn."""
import math

import pytest
import torch

import quantized_paged_kv_cache_gb300 as nk

import _ref
from _cases import compare

pytestmark = pytest.mark.gpu


def pool_of(k, v, P):
    L, H, D = k.shape
    n = -(-L // P) + 1
    pool = nk.KVPool.empty(n, P, H, D)
    pool.storage.fill_(0xFF)
    bt = torch.arange(n - 1, 0, -1, dtype=torch.int32, device="cuda").view(1, -1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    nk.kv_append(pool, bt, i32([0]), i32([0, L]), k.bfloat16(), v.bfloat16())
    return pool, bt


@pytest.mark.parametrize("W,S", [(100, 5), (1, 0), (77, 33)])
@pytest.mark.parametrize("D,P,Hq,H,T", [(256, 64, 24, 4, 1), (256, 64, 24, 4, 4), (256, 64, 30, 5, 5), (128, 16, 16, 2, 1),
                                        (128, 64, 16, 2, 2), (64, 32, 8, 8, 3), (256, 128, 12, 2, 1)])
def test_hidden_keys_leave_no_trace(D, P, Hq, H, T, W, S):
    L, scale = 500, 1 / math.sqrt(D)
    first = L - T - W + 1  # the first key that the first column's window holds
    g = torch.Generator(device="cuda").manual_seed(13)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    k, v, q = r(L, H, D), r(L, H, D), r(1, T, Hq, D).bfloat16()
    ctx, status = torch.tensor([L], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(pool, bt):
        return [nk.paged_window_attn(pool, q, bt, ctx, scale, L, W, sinks=S, status=status, num_ctas=n) for n in (0, 1)]

    pool, bt = pool_of(k, v, P)
    want = run(pool, bt)
    ref = _ref.attention(pool.storage, pool.num_pages, H, P, D, bt, [L], [T], q[0], scale, W, S).cpu().numpy()
    for o in want:
        compare(o, ref, "plain")
    for e in (16, 24, 60, 100):
        for x in (k, v):
            x[S:first] *= 2.0 ** e
            for o, w in zip(run(*pool_of(k, v, P)), want):
                assert torch.equal(o, w), f"hidden rows of 2^{e}"
            x[S:first] *= 2.0 ** -e
    n, sc = P * D, P * (D // 64) * 4
    for value in (float("inf"), float("-inf"), float("nan")):
        for a in (n, 2 * n + sc):  # the scales of K, of V
            pool, bt = pool_of(k, v, P)
            x = pool.storage.view(pool.num_pages, H, -1)[..., a:a + sc].view(torch.float32).unflatten(-1, (P, D // 64))
            for pos in range(S, first):
                x[int(bt[0, pos // P]), :, pos % P] = value
            for o, w in zip(run(pool, bt), want):
                assert torch.equal(o, w), f"hidden scales of {value}"
    assert int(status.item()) == 0
