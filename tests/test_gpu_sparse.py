"""Page bounds, page selection and attention over lists of pages
(nk_page_bounds, nk_page_select, nk_paged_sparse_attn) against plain forms:
bounds and selections bit for bit, attention to the decode calls' tolerances."""
import numpy as np
import pytest
import torch

import quantized_paged_kv_cache_gb300 as nk
from quantized_paged_kv_cache_gb300 import workloads as wl

import _long_ref as ref
from _cases import build, compare

pytestmark = pytest.mark.gpu

SHAPES = [
    # name, B, T, Hq, Hkv, D, P, ctx_lens
    ("t1_d256", 3, 1, 24, 4, 256, 64, [1, 700, 4099]),
    ("t4_d256", 2, 4, 24, 4, 256, 64, [4, 3001]),
    ("t16_d256", 2, 16, 24, 4, 256, 64, [16, 1500]),
    ("t1_d128_p16", 5, 1, 16, 2, 128, 16, [1, 15, 16, 17, 900]),
    ("t3_d64_p32", 2, 3, 8, 8, 64, 32, [1000, 50]),
    ("t2_d128_p128", 2, 2, 6, 2, 128, 128, [1300, 129]),
    ("t5_d64_p48", 3, 5, 10, 2, 64, 48, [5, 500, 49]),
    ("g14_d256", 1, 2, 14, 1, 256, 16, [777]),
    ("g48_d64", 1, 2, 48, 1, 64, 16, [300]),
]
IDS = [s[0] for s in SHAPES]


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def make(shape, seed=51, fill=0xFF, spare=2):
    name, B, T, Hq, Hkv, D, P, lens = shape
    w = wl.custom(name, B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, P=P, ctx_lens=lens, seed=seed,
                  num_pages=sum(-(-L // P) for L in lens) + spare, outlier_channels=2, outlier_scale=8.0)
    c = build(w, fill=fill, oracle_pool=False)
    c.status = i32([0])
    return c


def made_bounds(c):
    w = c.w
    b = nk.PageBounds.empty(c.pool)
    nk.page_bounds(c.pool, b, c.bt, i32([0] * w.B), i32(np.cumsum([0] + list(w.ctx_lens))), status=c.status)
    return b


def check_bounds(c, b, start, end, untouched):
    w = c.w
    kc, ks = ref.keys(c.pool.storage, w.num_pages, w.Hkv, w.P, w.D)
    codes, scales = b.codes().cpu().numpy(), b.scales().cpu().numpy()
    assert np.array_equal(b.values().cpu().numpy(), codes.astype(np.float32) * scales[..., None, None], equal_nan=True)
    left = np.ones(w.num_pages, bool)
    for s, (a, e) in enumerate(zip(start, end)):
        for i in range(a // w.P, -(-e // w.P) if e > a else 0):
            page = int(c.bt_cpu[s, i])
            want, sc = ref.bounds(kc, ks, page, min(w.P, e - i * w.P))
            assert np.array_equal(codes[page], want) and np.array_equal(scales[page], sc), (s, i)
            left[page] = False
    assert np.array_equal(codes[left], untouched[0][left]) and np.array_equal(scales[left], untouched[1][left])


# pages that the sparse attention has no kernel for, or that end inside a copy; more items than blocks
BOUNDS = SHAPES + [("d256_p256", 1, 1, 8, 2, 256, 256, [1300]), ("d64_p80", 2, 1, 4, 2, 64, 80, [999, 81]),
                   ("many", 5, 1, 8, 8, 128, 16, [900, 333, 16, 1, 700]), ("many_d256", 2, 1, 4, 4, 256, 64, [6000, 4001])]


@pytest.mark.parametrize("shape", BOUNDS, ids=[s[0] for s in BOUNDS])
def test_bounds(shape):
    c = make(shape)
    w = c.w
    before = (np.zeros((w.num_pages, w.Hkv, 2, w.D), np.int8), np.zeros((w.num_pages, w.Hkv), np.float32))
    check_bounds(c, made_bounds(c), [0] * w.B, w.ctx_lens, before)
    # a later step's pages only, the others as they were; one sequence that brings nothing
    b = nk.PageBounds.empty(c.pool)
    b.storage.fill_(0x11)
    before = b.codes().cpu().numpy().copy(), b.scales().cpu().numpy().copy()
    start = [max(0, L - 1 - 7 * i) for i, L in enumerate(w.ctx_lens)]
    start[-1] = w.ctx_lens[-1] if w.B > 1 else start[-1]
    new = [L - s for L, s in zip(w.ctx_lens, start)]
    g = torch.cuda.CUDAGraph()
    args = i32(start), i32(np.cumsum([0] + new))
    with torch.cuda.graph(g):
        nk.page_bounds(c.pool, b, c.bt, *args, status=c.status)
    g.replay()
    check_bounds(c, b, start, w.ctx_lens, before)
    assert int(c.status.item()) == 0


def test_bounds_of_odd_keys_and_bad_data():
    c = make(("odd", 2, 1, 4, 2, 64, 16, [40, 33]))
    w = c.w
    raw = c.pool.storage.view(w.num_pages, w.Hkv, -1)
    scales = raw[..., 16 * 64:16 * 64 + 64].view(torch.float32)
    page = int(c.bt_cpu[0, 1])
    raw[int(c.bt_cpu[0, 0]), :, :16 * 64] = 0  # a page of zeros: scale 1
    scales[page, 0, 3], scales[page, 1, 5] = float("nan"), float("inf")  # these keys count as zeros
    b = made_bounds(c)
    before = (np.zeros((w.num_pages, w.Hkv, 2, w.D), np.int8), np.zeros((w.num_pages, w.Hkv), np.float32))
    check_bounds(c, b, [0, 0], w.ctx_lens, before)
    assert b.scales()[int(c.bt_cpu[0, 0])].tolist() == [1.0, 1.0]
    assert int(c.status.item()) == nk.NK_DEVFLAG_RANGE
    for start, cu, bt, flag in (([-1, 0], [0, 5, 38], c.bt, nk.NK_DEVFLAG_BAD_POS), ([0, 0], [0, -3, 30], c.bt, nk.NK_DEVFLAG_BAD_POS),
                                ([48, 0], [0, 1, 34], c.bt, nk.NK_DEVFLAG_BAD_POS), ([0, 0], [0, 1, 34], None, nk.NK_DEVFLAG_BAD_PAGE)):
        c.status.zero_()
        b.storage.zero_()
        table = c.bt[:, :3].contiguous()
        if bt is None:
            table[0, 0] = w.num_pages
        nk.page_bounds(c.pool, b, table, i32(start), i32(cu), status=c.status)
        assert int(c.status.item()) == flag
        assert not b.scales()[c.bt_cpu[0, :3].long()].any()  # the refused sequence's pages
        assert b.scales()[int(c.bt_cpu[1, 0])].all()
    nk.page_bounds(c.pool, b, c.bt[:0].contiguous(), i32([]), i32([0]))  # no sequences


def selections(c, k, sinks, recent, bounds, **kw):
    w = c.w
    return nk.page_select(bounds, kw.pop("q", c.q), kw.pop("bt", c.bt), c.ctx, w.P, w.max_ctx, k, sink_pages=sinks, recent_pages=recent,
                          status=c.status, **kw)


def expected(c, k, sinks, recent, bounds, q=None, bt=None):
    w = c.w
    return ref.select(bounds.codes().cpu().numpy(), bounds.scales().cpu().numpy(), (c.q if q is None else q).double().cpu().numpy(),
                      (c.bt_cpu if bt is None else bt.cpu()).numpy(), w.ctx_lens, w.P, k, sinks, recent)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_select(shape):
    c = make(shape)
    b = made_bounds(c)
    for k, sinks, recent in ((1, 0, 1), (2, 1, 1), (3, 0, 1), (7, 2, 3), (9, 1, 2), (200, 1, 1)):
        got = selections(c, k, sinks, recent, b)
        assert np.array_equal(got.cpu().numpy(), expected(c, k, sinks, recent, b)), (k, sinks, recent)
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("pages", [130, 2049, 9000, 17000])
def test_select_from_many_pages(pages):
    """More pages than a block's bins, than a round of blocks takes, than stay in shared memory."""
    B, T, Hq, Hkv, D, P = 2, 2, 4, 2, 64, 16
    gen = torch.Generator(device="cuda")
    gen.manual_seed(pages)
    n = [pages, pages // 3]
    num = sum(n) + 1
    table = torch.full((B, pages), -1, dtype=torch.int32, device="cuda")
    perm = torch.randperm(num, generator=gen, device="cuda").to(torch.int32)
    table[0], table[1, :n[1]] = perm[:n[0]], perm[n[0]:n[0] + n[1]]
    b = nk.PageBounds(torch.empty(num * Hkv * (2 * D + 4), dtype=torch.uint8, device="cuda"), num, Hkv, D)
    b.codes().copy_(torch.randint(-127, 128, (num, Hkv, 2, D), generator=gen, device="cuda"))
    b.scales().copy_(torch.rand((num, Hkv), generator=gen, device="cuda") ** 4)
    q = torch.randn((B, T, Hq, D), generator=gen, device="cuda").to(torch.bfloat16)
    ctx = [x * P - 3 for x in n]
    for k, sinks, recent in ((64, 1, 2), (1000, 0, 1)):
        got = nk.page_select(b, q, table, i32(ctx), P, max(ctx), k, sink_pages=sinks, recent_pages=recent).cpu().numpy()
        want = ref.select(b.codes().cpu().numpy(), b.scales().cpu().numpy(), q.double().cpu().numpy(), table.cpu().numpy(), ctx, P, k, sinks, recent)
        assert np.array_equal(got, want)


@pytest.mark.parametrize("what", ["equal", "few_values", "huge_and_tiny", "negative", "zero_queries", "odd_queries", "bad_page", "odd_bounds"])
def test_select_ties_and_ranges(what):
    c = make(("ties", 2, 2, 6, 2, 128, 16, [1500, 900]))
    w = c.w
    b = made_bounds(c)
    codes, scales = b.codes(), b.scales()
    q, bt = c.q.clone(), c.bt.clone()
    rng = torch.Generator().manual_seed(3)
    if what == "equal":
        codes[:] = codes[:1].clone()
        scales.fill_(0.37)
    elif what == "few_values":
        pick = torch.randint(0, 3, (w.num_pages,), generator=rng).cuda()
        codes[:], scales[:] = codes[:3][pick].clone(), scales[:3][pick].clone()
    elif what == "huge_and_tiny":
        scales.copy_(2.0 ** torch.randint(-140, 120, tuple(scales.shape), generator=rng).double())
    elif what == "negative":
        codes[:, :, 0], codes[:, :, 1] = -codes[:, :, 0].abs(), codes[:, :, 1].abs()
    elif what == "zero_queries":
        q.zero_()
    elif what == "odd_queries":
        q[0, 0, 1, 5], q[1, 1, 4, 7] = float("nan"), float("inf")
    elif what == "bad_page":
        bt[0, 5], bt[1, 30] = -1, w.num_pages
    else:
        scales[int(c.bt_cpu[0, 9])] = float("nan")
        scales[int(c.bt_cpu[0, 11])] = float("inf")
    for k, sinks, recent in ((5, 0, 1), (40, 2, 3)):
        got = selections(c, k, sinks, recent, b, q=q, bt=bt)
        assert np.array_equal(got.cpu().numpy(), expected(c, k, sinks, recent, b, q=q, bt=bt)), (k, sinks, recent)
    assert int(c.status.item()) == (nk.NK_DEVFLAG_BAD_PAGE if what == "bad_page" else 0)


def test_select_captured_and_on_another_stream():
    c = make(("graph", 2, 3, 8, 2, 128, 16, [1200, 400]))
    w, b = c.w, made_bounds(c)
    want = expected(c, 9, 1, 2, b)
    out, g = torch.empty((2, 3, 2, 9), dtype=torch.int32, device="cuda"), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        selections(c, 9, 1, 2, b, out=out)
        selections(c, 9, 1, 2, b, out=out)
    g.replay()
    g.replay()
    assert np.array_equal(out.cpu().numpy(), want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = selections(c, 9, 1, 2, b, stream=st)
    lists = nk.paged_sparse_attn(c.pool, c.q, c.bt, c.ctx, got, w.sm_scale, w.max_ctx, stream=st)
    st.synchronize()
    assert np.array_equal(got.cpu().numpy(), want)
    assert torch.equal(lists, nk.paged_sparse_attn(c.pool, c.q, c.bt, c.ctx, got, w.sm_scale, w.max_ctx))


def test_select_leaves_an_invalid_sequences_lists():
    c = make(("inv", 3, 2, 4, 2, 64, 16, [200, 300, 100]))
    b = made_bounds(c)
    want = expected(c, 6, 1, 1, b)
    c.ctx[1] = 1  # fewer than T
    out = torch.full((3, 2, 2, 6), -9, dtype=torch.int32, device="cuda")
    selections(c, 6, 1, 1, b, out=out)
    got = out.cpu().numpy()
    assert (got[1] == -9).all() and np.array_equal(got[[0, 2]], want[[0, 2]])
    assert int(c.status.item()) == nk.NK_DEVFLAG_BAD_CTX


def lists_of(c, k, rng, kind):
    """int32 [B][T][Hkv][k]: random pages that the token sees, in random order, with entries that name none between."""
    w = c.w
    out = np.full((w.B, w.T, w.Hkv, k), -1, np.int64)
    for b in range(w.B):
        for t in range(w.T):
            seen = (w.ctx_lens[b] - w.T + t) // w.P + 1
            for h in range(w.Hkv):
                if kind == "empty" and (b + t + h) % 2:
                    continue
                pick = rng.permutation(seen)[:min(seen, k)]
                if kind == "holes" and len(pick) > 1:
                    pick[rng.randint(len(pick))] = rng.choice([-1, -5, seen, 1 << 30])
                if kind == "sorted":
                    pick = np.sort(pick)
                out[b, t, h, :len(pick)] = pick
    return out


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("kind", ["sorted", "holes", "empty"])
def test_sparse_attention(shape, kind):
    c = make(shape)
    w = c.w
    rng = np.random.RandomState(5)
    for k in (1, 3, 20, 300):
        lists = lists_of(c, k, rng, kind)
        want = ref.sparse(c.pool.storage, w.num_pages, w.Hkv, w.P, w.D, c.bt_cpu.numpy(), w.ctx_lens, lists, c.q, w.sm_scale)
        for n in (0, 1, 5):
            got = nk.paged_sparse_attn(c.pool, c.q, c.bt, c.ctx, i32(lists), w.sm_scale, w.max_ctx, num_ctas=n, status=c.status)
            compare(got, want, f"{w.name} {kind} k={k} ctas={n}")
        assert torch.equal(got, nk.paged_sparse_attn(c.pool, c.q, c.bt, c.ctx, i32(lists), w.sm_scale, w.max_ctx, num_ctas=n))
        none = torch.from_numpy(~np.isin(lists, np.arange(1 << 20)).any(-1))
        if kind == "empty" and none.any():
            rows = got.view(w.B, w.T, w.Hkv, -1)[none.to("cuda")]
            assert not rows.any()
    assert int(c.status.item()) == 0


def test_sparse_attention_over_more_pages_than_a_cta_keeps():
    c = make(("far", 1, 1, 2, 1, 64, 16, [30000]))
    w = c.w
    lists = lists_of(c, 1700, np.random.RandomState(6), "holes")
    want = ref.sparse(c.pool.storage, w.num_pages, w.Hkv, w.P, w.D, c.bt_cpu.numpy(), w.ctx_lens, lists, c.q, w.sm_scale)
    for n in (1, 2, 0):
        compare(nk.paged_sparse_attn(c.pool, c.q, c.bt, c.ctx, i32(lists), w.sm_scale, w.max_ctx, num_ctas=n), want, f"ctas={n}")


def test_sparse_attention_reads_listed_pages_only():
    c = make(("listed", 2, 2, 8, 2, 128, 16, [400, 333]))
    w = c.w
    lists = lists_of(c, 4, np.random.RandomState(7), "sorted")
    want = nk.paged_sparse_attn(c.pool, c.q, c.bt, c.ctx, i32(lists), w.sm_scale, w.max_ctx)
    bt = c.bt.clone()
    for b in range(2):
        rest = np.setdiff1d(np.arange(bt.shape[1]), lists[b])
        bt[b, torch.from_numpy(rest).cuda()] = -1  # given back
    got = nk.paged_sparse_attn(c.pool, c.q, bt, c.ctx, i32(lists), w.sm_scale, w.max_ctx, status=c.status)
    assert torch.equal(got, want) and int(c.status.item()) == 0
    bt[0, int(lists[0, 0, 0, 0])] = w.num_pages
    nk.paged_sparse_attn(c.pool, c.q, bt, c.ctx, i32(lists), w.sm_scale, w.max_ctx, status=c.status)
    assert int(c.status.item()) == nk.NK_DEVFLAG_BAD_PAGE
    c.status.zero_()
    c.ctx[1] = w.max_ctx + 1
    got = nk.paged_sparse_attn(c.pool, c.q, c.bt, c.ctx, i32(lists), w.sm_scale, w.max_ctx, status=c.status)
    assert torch.equal(got[0], want[0]) and int(c.status.item()) == nk.NK_DEVFLAG_BAD_CTX


def test_a_list_of_everything_is_the_whole_context():
    c = make(("all", 2, 4, 24, 4, 256, 64, [900, 333]))
    w = c.w
    lists = selections(c, 20, 1, 1, made_bounds(c))
    got = nk.paged_sparse_attn(c.pool, c.q, c.bt, c.ctx, lists, w.sm_scale, w.max_ctx)
    compare(got, nk.paged_decode_attn(c.pool, c.q, c.bt, c.ctx, w.sm_scale, w.max_ctx).double().cpu().numpy(), "all pages")
