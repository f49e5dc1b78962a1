"""Keys in the blocks that nk_paged_chunk_attn works on but that no token of the chunk sees (before every window and behind
the sinks): their K and V, of any size or not finite, leave no trace and set no flag."""
import math

import pytest
import torch

import quantized_paged_kv_cache_gb300 as nk

import _ref
from test_gpu_chunk import check
from test_gpu_window_hidden import pool_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("W,S", [(100, 5), (1, 0), (77, 33), (64, 64)])
@pytest.mark.parametrize("D,P,Hq,H,T", [(256, 64, 24, 4, 20), (128, 16, 16, 2, 7), (128, 128, 6, 2, 40), (64, 48, 8, 8, 100)])
def test_hidden_keys_leave_no_trace(D, P, Hq, H, T, W, S):
    L, scale = 500, 1 / math.sqrt(D)  # (one tile of rows a kv-head)
    first = L - T - W + 1  # the first key that the first token's window holds
    g = torch.Generator(device="cuda").manual_seed(14)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    k, v, q = r(L, H, D), r(L, H, D), r(T, Hq, D).bfloat16()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ctx, cu, status = i32([L]), i32([0, T]), i32([0])

    def run(pool, bt):
        return [nk.paged_chunk_attn(pool, q, cu, bt, ctx, scale, L, window=W, sinks=S, status=status, num_ctas=n) for n in (0, 1)]

    pool, bt = pool_of(k, v, P)
    want = run(pool, bt)
    ref = _ref.attention(pool.storage, pool.num_pages, H, P, D, bt, [L], [T], q, scale, W, S)
    for o in want:
        check(o, ref, "plain")
    for e in (8, 20, 60, 100):
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


def test_a_later_token_that_is_not_finite_leaves_the_tiles_before_it():
    """Two tiles of 32 tokens (G = 4): what the last token brought is no business of the first tile, nor its exponents'."""
    H, D, P, L, T = 2, 128, 64, 64, 64
    g = torch.Generator(device="cuda").manual_seed(15)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    k, v, q = r(L, H, D), r(L, H, D), r(T, 4 * H, D).bfloat16()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    args = (i32([0, T]),), (i32([L]), 1 / math.sqrt(D), L)

    def run(k, v):
        pool, bt = pool_of(k, v, P)
        return nk.paged_chunk_attn(pool, q, *args[0], bt, *args[1])

    want = run(k, v)
    k[33:] *= 2.0 ** 30
    v[33:] *= 2.0 ** 30
    v[40] = float("inf")
    assert torch.equal(run(k, v)[:32], want[:32])


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_query_that_is_not_finite_is_nan_however_the_work_is_split(value):
    L, T, Hq, H, D = 2000, 9, 8, 2, 128
    g = torch.Generator(device="cuda").manual_seed(16)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    pool, bt = pool_of(r(L, H, D), r(L, H, D), 64)
    q = r(T, Hq, D).bfloat16()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ctx, cu = i32([L]), i32([0, T])
    for n in (1, 2, 7, 0):
        status = i32([0])
        run = lambda q: nk.paged_chunk_attn(pool, q, cu, bt, ctx, 0.1, L, num_ctas=n, status=status)  # noqa: B023, E731
        want = run(q)
        bad = q.clone()
        bad[5, 3] = value
        out = run(bad)
        torch.cuda.synchronize()
        assert int(status.item()) == nk.NK_DEVFLAG_RANGE
        assert torch.isnan(out[5, 3]).all(), f"{n} CTAs"
        out[5, 3] = want[5, 3]
        assert torch.equal(out, want), "the other rows"
