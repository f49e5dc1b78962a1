"""Page weights (nk_page_weights) where a query row sees no key: the pages that it could see first lie outside the pool. Such
a row draws nothing, and the other rows' weights stand; against a plain form in 64 bits."""
import numpy as np
import pytest
import torch

import quantized_paged_kv_cache_gb300 as nk
from quantized_paged_kv_cache_gb300 import workloads as wl

import _ref
from _cases import build

pytestmark = pytest.mark.gpu

SHAPES = [
    # name, B, T, Hq, Hkv, D, P, ctx_lens, logical pages of the first sequence that are none
    ("tc_d64", 2, 16, 8, 2, 64, 16, [30, 100], [0]),              # 64 rows: tcgen05; rows 0 and 1 see page 0 alone
    ("tc_d256_p64", 2, 16, 7, 1, 256, 64, [70, 300], [0]),        # rows 0 to 9
    ("tc_two_chunks", 1, 16, 14, 1, 128, 16, [45], [0, 1]),       # 224 rows; rows 0 to 2
    ("tc_shared_tile", 2, 16, 4, 1, 128, 32, [47, 64], [0]),      # rows 0 only
    ("mma_one_tile", 2, 4, 2, 1, 256, 16, [18, 40], [0]),         # rows 0 and 1 of 8
    ("mma_tiles", 2, 16, 4, 2, 128, 16, [30, 77], [0]),           # 32 rows
    ("mma_p48", 1, 5, 6, 1, 64, 48, [50], [0]),
    ("mma_long", 2, 8, 6, 1, 128, 16, [2003, 1500], list(range(125))),  # several CTAs; rows 0 to 4
]


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def case(shape):
    name, B, T, Hq, Hkv, D, P, lens, gone = shape
    c = build(wl.custom(name, B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, P=P, ctx_lens=lens, seed=83,
                        num_pages=sum(-(-L // P) for L in lens) + 2), fill=0xFF, oracle_pool=False)
    c.status = i32([0])
    c.table = c.bt.clone()
    c.table[0, gone] = i32([(-1, c.w.num_pages)[i % 2] for i in range(len(gone))])
    return c


def plain(c, table):
    """fp64 [num_pages][Hkv], NaN for pages that the batch does not hold, and how many rows see no key."""
    w = c.w
    K = _ref.dequantized(c.pool.storage, w.num_pages, w.Hkv, w.P, w.D)[0].cpu().numpy()
    q, table = c.q.double().cpu().numpy(), table.cpu().numpy()
    out, G, none = np.full((w.num_pages, w.Hkv), np.nan), w.Hq // w.Hkv, 0
    for b, L in enumerate(w.ctx_lens):
        pages = -(-L // w.P)
        good = [i for i in range(pages) if 0 <= table[b, i] < w.num_pages]
        for h in range(w.Hkv):
            for i in good:
                out[table[b, i], h] = 0.0
            for t in range(w.T):
                pos = L - w.T + t
                keys = [(i, K[table[b, i], h, :min(w.P, pos + 1 - i * w.P)]) for i in good if i * w.P <= pos]
                if not keys:
                    none += 1
                    continue
                s = q[b, t, h * G:(h + 1) * G] @ np.concatenate([k for _, k in keys]).T * w.sm_scale
                e = np.exp(s - s.max(-1, keepdims=True))
                mass = (e / e.sum(-1, keepdims=True)).sum(0)
                at = 0
                for i, k in keys:
                    out[table[b, i], h] += mass[at:at + len(k)].sum()
                    at += len(k)
    return out, none


def check(got, want, before):
    """Held to 1e-4 of a weight, and 1e-6 beside it: a score is the exponential's argument, some 24 roundings of 2^-23 of what
    its products' sizes add up to, under 20 for unit queries and keys (6e-5 of the weight at worst)."""
    got, held = got.double().cpu().numpy(), ~np.isnan(want)
    assert np.isfinite(got[held]).all()
    assert (np.abs(got - want)[held] <= 1e-4 * want[held] + 1e-6).all()
    assert (got[~held] == before).all()


@pytest.mark.parametrize("shape", SHAPES, ids=[s[0] for s in SHAPES])
def test_rows_that_see_no_key_draw_nothing(shape):
    c = case(shape)
    w = c.w
    want, none = plain(c, c.table)
    assert none > 0
    out = torch.full((w.num_pages, w.Hkv), -3.0, device="cuda")
    nk.page_weights(c.pool, c.q, c.table, c.ctx, w.sm_scale, w.max_ctx, out, status=c.status)
    assert int(c.status.item()) == nk.NK_DEVFLAG_BAD_PAGE
    check(out, want, -3.0)
    # added in place to what stands there
    once = out.clone()
    for n in (2, 3):
        nk.page_weights(c.pool, c.q, c.table, c.ctx, w.sm_scale, w.max_ctx, out, prior=out)
        check(out, n * want, -3.0)
    held = torch.from_numpy(~np.isnan(want)).cuda()
    seen = i32([0] * w.B)  # nothing has an earlier sum: the first result again, bit for bit
    nk.page_weights(c.pool, c.q, c.table, c.ctx, w.sm_scale, w.max_ctx, out, prior=out, seen=seen)
    assert torch.equal(out[held], once[held])


@pytest.mark.parametrize("T,Hq", [(1, 2), (4, 12), (16, 12)])
def test_a_sequence_of_no_page_in_the_pool(T, Hq):
    c = case(("none", 2, T, Hq, 2, 64, 16, [40, 50], [0, 1, 2]))
    w = c.w
    want, none = plain(c, c.table)
    out = torch.full((w.num_pages, w.Hkv), -3.0, device="cuda")
    nk.page_weights(c.pool, c.q, c.table, c.ctx, w.sm_scale, w.max_ctx, out, status=c.status)
    assert none == 2 * T and int(c.status.item()) == nk.NK_DEVFLAG_BAD_PAGE
    check(out, want, -3.0)


@pytest.mark.parametrize("T,Hq", [(1, 4), (4, 12), (16, 8)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_an_infinite_query_spoils_its_kv_head_and_no_other(T, Hq, sign):
    """Every score of the row is the same infinity: minus infinity alone leaves no key of weight, and is no empty row."""
    c = case(("inf", 2, T, Hq, 2, 64, 16, [100, 60], []))
    w = c.w
    codes = c.pool.storage.view(w.num_pages, w.Hkv, -1)[..., :16 * 64].view(torch.int8).view(w.num_pages, w.Hkv, 16, 64)
    codes[..., 5] = 50
    good, out = torch.zeros((w.num_pages, w.Hkv), device="cuda"), torch.zeros((w.num_pages, w.Hkv), device="cuda")
    nk.page_weights(c.pool, c.q, c.bt, c.ctx, w.sm_scale, w.max_ctx, good)
    q = c.q.clone()
    q[0, T - 1, Hq - 1, 5] = sign * float("inf")
    nk.page_weights(c.pool, q, c.bt, c.ctx, w.sm_scale, w.max_ctx, out)
    pages = c.bt_cpu[0, :7].long()
    assert out[pages, 1].isnan().all()
    assert torch.equal(out[pages, 0], good[pages, 0])
    other = c.bt_cpu[1, :4].long()
    assert torch.equal(out[other], good[other])
