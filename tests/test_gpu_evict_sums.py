"""The order of evictions (nk_evict_pages) over weights that spread over many binades: the sums over the kv-heads do not depend
on the heads' order, and what 55 bits tell apart is told apart. Against exact fractions."""
import numpy as np
import pytest
import torch

import quantized_paged_kv_cache_gb300 as nk

import _long_ref as ref

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def evicted(w, keep, sinks=0, recent=1, plain=None):
    """One sequence over all pages of `w`, in order, and a last one that stays in any case."""
    n = len(w)
    table, ctx = np.arange(n)[None], [16 * n]
    want, lens, freed = ref.evict(w if plain is None else plain, table, ctx, 16, keep, sinks, recent)
    tb, new, lst, count = i32(table), i32([0]), i32([-7] * (n + 1)), i32([0])
    nk.evict_pages(16, torch.from_numpy(np.ascontiguousarray(w, np.float32)).cuda(), tb, i32(ctx), keep, new, lst, count,
                   sink_pages=sinks, recent_pages=recent)
    assert new.tolist() == lens and count.tolist() == [len(freed)]
    return lst.tolist()[:len(freed)], freed, tb.cpu().numpy(), want


@pytest.mark.parametrize("first,second", [
    ([1.178e-5, 0.71719, 0.058709, 3.9025e-8], [3.9025e-8, 0.058709, 1.178e-5, 0.71719]),  # the same numbers: the lower page stays
    ([3.9025e-8, 0.058709, 1.178e-5, 0.71719], [1.178e-5, 0.71719, 0.058709, 3.9025e-8]),
    ([1, 2.0 ** -26, 0, 0], [1, 2.0 ** -26, 2.0 ** -52, 0]),  # the higher page is worth more
    ([1, 2.0 ** -25, 0], [1, 2.0 ** -25, 2.0 ** -50]),
    ([2.0 ** -50, 2.0 ** -25, 1], [2.0 ** -25, 1, 2.0 ** -50]),
    ([1, 1, -2.0 ** -53], [1, 1, 0]),
    ([-1, -2.0 ** -52, 0], [-1, -2.0 ** -53, 0]),
    ([2.0 ** -149, 0, 0], [2.0 ** -149, 2.0 ** -149, 0]),
    ([2.0 ** 127, 2.0 ** 127, 0], [2.0 ** 127, 2.0 ** 127, 2.0 ** 80]),
    ([1, -1, 0], [0, 0, -0.0]),
])
def test_two_pages(first, second):
    w = np.float32([first, second, [0] * len(first)])
    got, want, tb, table = evicted(w, 2)
    assert got == want and np.array_equal(tb, table)


@pytest.mark.parametrize("Hkv", [1, 2, 3, 4, 5, 8, 12])
def test_the_order_of_heads_changes_nothing(Hkv):
    """Weights within 2^-24 of their page's largest, so that no sum needs more than 24 + 24 + 4 bits; every page comes
    twice, its heads in another order."""
    rng = np.random.RandomState(Hkv)
    n = 1000
    w = np.exp(-16 * rng.rand(n, Hkv)).astype(np.float32)
    both = np.empty((2 * n + 1, Hkv), np.float32)
    both[0:2 * n:2] = w
    both[1:2 * n:2] = w[:, rng.permutation(Hkv)[::-1]]
    both[2 * n] = 0
    for keep in (2, 702, 1501):  # (odd numbers of pages beside the last: a pair is parted)
        got, want, tb, table = evicted(both, keep)
        assert got == want and np.array_equal(tb, table), keep


def test_what_is_not_finite():
    inf, nan, big = np.float32("inf"), np.float32("nan"), np.float32(3e38)
    # infinities count as 2^128, a page with a NaN is the first to go
    w = np.float32([[big, 0], [inf, 0], [nan, big], [-inf, -inf], [-big, -big], [nan, inf], [0, 0]])
    plain = w.astype(np.float64)
    plain[np.isinf(plain)] = np.sign(plain[np.isinf(plain)]) * 2.0 ** 128
    plain[np.isnan(w).any(1)] = -2.0 ** 140
    for keep in range(2, 7):
        got, want, tb, table = evicted(w, keep, plain=plain)
        assert got == want and np.array_equal(tb, table), keep
