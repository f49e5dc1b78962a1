"""Attention weights of pages and eviction by them (nk_page_weights,
nk_evict_pages) against plain forms, and a serving step of all the operators
over long caches together."""
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
    ("t2_d128_p256", 2, 2, 6, 2, 128, 256, [1300, 129]),
    ("t5_d64_p48", 3, 5, 10, 2, 64, 48, [5, 500, 49]),
    ("t16_g14", 1, 16, 14, 1, 256, 16, [777]),
    ("t16_g7", 40, 16, 7, 1, 64, 16, [16 + 5 * i for i in range(40)]),
]
IDS = [s[0] for s in SHAPES]


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def make(shape, seed=61, spare=2, **kw):
    name, B, T, Hq, Hkv, D, P, lens = shape
    w = wl.custom(name, B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, P=P, ctx_lens=lens, seed=seed,
                  num_pages=sum(-(-L // P) for L in lens) + spare, outlier_channels=2, outlier_scale=8.0, **kw)
    c = build(w, fill=0xFF, oracle_pool=False)
    c.status = i32([0])
    return c


def check_weights(c, got, want, before, prior=None, what="", tol=1e-4):
    """A weight is the exponential of a score. A score is the sum of D <= 256 products, 16 a step of the tensor cores and a
    group's scale every four steps: some 24 roundings, each at most 2^-23 of what the products' sizes add up to, about 20
    here (300 with the two outlier channels, times sm_scale), so 24 * 20 * 2^-23 = 6e-5 of the weight at worst. The
    exponentials and sums add a few 2^-22. Held: 1e-4 of the weight (more as the scale is larger), and 1e-6 beside it for
    sums of tiny ones."""
    w = c.w
    got = got.double().cpu().numpy()
    touched = np.zeros((w.num_pages, w.Hkv), bool)
    for (page, h), m in want.items():
        touched[page, h] = True
        if prior is not None:
            m = m + prior.get((page, h), 0.0)
        assert abs(got[page, h] - m) <= tol * m + 1e-6, (what, page, h, got[page, h], m)
    assert np.array_equal(got[~touched], before.double().cpu().numpy()[~touched]), what


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_weights(shape):
    c = make(shape)
    w = c.w
    want = ref.weights(c.pool.storage, w.num_pages, w.Hkv, w.P, w.D, c.bt_cpu.numpy(), w.ctx_lens, c.q, w.sm_scale)
    before = torch.full((w.num_pages, w.Hkv), -7.0, device="cuda")
    out = before.clone()
    got = nk.page_weights(c.pool, c.q, c.bt, c.ctx, w.sm_scale, w.max_ctx, out, status=c.status)
    assert got is out
    check_weights(c, got, want, before, what="fresh")
    for b in range(w.B):  # every row's weights sum to 1
        n = -(-w.ctx_lens[b] // w.P)
        total = got[c.bt[b, :n].long()].double().sum(0).cpu().numpy()
        assert np.allclose(total, w.T * (w.Hq // w.Hkv), rtol=1e-5)
    # accumulated in place, captured and replayed; pages past `seen` start anew whatever they hold
    seen = [max(0, L - 40 * i - 3) for i, L in enumerate(w.ctx_lens)]
    acc = torch.rand((w.num_pages, w.Hkv), device="cuda") + 0.5
    first = acc.clone()
    prior = {}
    for b in range(w.B):
        for i in range(-(-seen[b] // w.P)):
            for h in range(w.Hkv):
                prior[int(c.bt_cpu[b, i]), h] = float(first[int(c.bt_cpu[b, i]), h])
    seen_dev, g = i32(seen), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nk.page_weights(c.pool, c.q, c.bt, c.ctx, w.sm_scale, w.max_ctx, acc, prior=acc, seen=seen_dev, status=c.status)
    g.replay()
    check_weights(c, acc, want, first, prior, what="in place")
    again = torch.empty_like(first)
    again.copy_(first)
    nk.page_weights(c.pool, c.q, c.bt, c.ctx, w.sm_scale, w.max_ctx, again, prior=first, seen=seen_dev)
    assert torch.equal(again, acc)  # the same in every run, in place or not
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("shape", [("many_t1", 2, 1, 6, 2, 64, 16, [100000, 60001]), ("many_t16", 1, 16, 8, 2, 64, 64, [200003]),
                                   ("many_t16_p16", 1, 16, 8, 1, 64, 16, [99999]), ("many_t5_p128", 3, 5, 12, 2, 128, 128, [40000, 30001, 77]),
                                   ("many_t16_p32", 2, 16, 14, 1, 64, 32, [70000, 12345]),
                                   ("many_short", 300, 4, 16, 2, 64, 32, [4 + (37 * i) % 190 for i in range(300)]),
                                   ("many_t16_p48", 1, 16, 8, 2, 128, 48, [30001]), ("many_t16_p80", 1, 16, 8, 1, 64, 80, [25003]),
                                   ("many_t16_p256", 1, 16, 12, 2, 256, 256, [20011]), ("many_t4_p80", 1, 4, 12, 2, 128, 80, [20001]),
                                   ("one_tile_each", 700, 2, 26, 2, 64, 64, [2 + (11 * i) % 63 for i in range(700)])], ids=lambda s: s[0])
def test_weights_of_long_contexts(shape):
    """Dozens of pages a CTA, so that every ring goes round; segments that end inside a CTA's range."""
    c = make(shape)
    w = c.w
    want = ref.weights(c.pool.storage, w.num_pages, w.Hkv, w.P, w.D, c.bt_cpu.numpy(), w.ctx_lens, c.q, w.sm_scale)
    out = torch.zeros((w.num_pages, w.Hkv), device="cuda")
    got = nk.page_weights(c.pool, c.q, c.bt, c.ctx, w.sm_scale, w.max_ctx, out, status=c.status)
    assert int(c.status.item()) == 0
    check_weights(c, got, want, torch.zeros_like(out))


@pytest.mark.parametrize("q_scale,k_scale", [(2.0 ** 60, 2.0 ** -60), (2.0 ** -80, 2.0 ** 80), (2.0 ** -30, 1.0)])
def test_weights_far_off_unit_scale(q_scale, k_scale):
    c = make(("range", 2, 3, 6, 2, 128, 16, [200, 77]), q_scale=q_scale, k_scale=k_scale)
    w = c.w
    want = ref.weights(c.pool.storage, w.num_pages, w.Hkv, w.P, w.D, c.bt_cpu.numpy(), w.ctx_lens, c.q, w.sm_scale)
    out = torch.zeros((w.num_pages, w.Hkv), device="cuda")
    check_weights(c, nk.page_weights(c.pool, c.q, c.bt, c.ctx, w.sm_scale, w.max_ctx, out), want, torch.zeros_like(out))


@pytest.mark.parametrize("T", [1, 16])
@pytest.mark.parametrize("scale", [0.0, -0.07, 0.5])
def test_weights_of_any_scale(T, scale):
    c = make(("scale", 2, T, 10, 2, 128, 32, [300, 77]))
    w = c.w
    want = ref.weights(c.pool.storage, w.num_pages, w.Hkv, w.P, w.D, c.bt_cpu.numpy(), w.ctx_lens, c.q, scale)
    out = torch.zeros((w.num_pages, w.Hkv), device="cuda")
    nk.page_weights(c.pool, c.q, c.bt, c.ctx, scale, w.max_ctx, out)
    check_weights(c, out, want, torch.zeros_like(out), tol=4e-4 if scale == 0.5 else 1e-4)


@pytest.mark.parametrize("T,Hq", [(2, 4), (16, 8)])
def test_weights_of_odd_data(T, Hq):
    c = make(("odd", 3, T, Hq, 2, 64, 16, [100, 60, 30]))
    w = c.w
    plain = torch.zeros((w.num_pages, w.Hkv), device="cuda")
    nk.page_weights(c.pool, c.q, c.bt, c.ctx, w.sm_scale, w.max_ctx, plain)
    pages = [c.bt_cpu[b, :-(-w.ctx_lens[b] // 16)].long() for b in range(3)]
    # a query that is not finite spoils its own kv-head's pages and no others
    for bad in (float("nan"), float("inf")):
        q, out = c.q.clone(), torch.zeros_like(plain)
        q[0, 1, Hq - 1, 2] = bad
        nk.page_weights(c.pool, q, c.bt, c.ctx, w.sm_scale, w.max_ctx, out)
        assert out[pages[0], 1].isnan().all()
        assert torch.equal(out[pages[0], 0], plain[pages[0], 0]) and torch.equal(out[pages[1]], plain[pages[1]])
    # lengths that are refused, a page outside the pool (it draws nothing), a scale past the length
    ctx, bt, out = c.ctx.clone(), c.bt.clone(), torch.full_like(plain, -3.0)
    ctx[1] = T - 1
    bt[2, 0] = w.num_pages
    nk.page_weights(c.pool, c.q, bt, ctx, w.sm_scale, w.max_ctx, out, status=c.status)
    assert int(c.status.item()) == nk.NK_DEVFLAG_BAD_CTX | nk.NK_DEVFLAG_BAD_PAGE
    assert (out[pages[1]] == -3).all()
    # (the CTAs' ranges are others without the sequence, so a row's log-sum is joined in another order: a few 2^-22 of it)
    assert torch.allclose(out[pages[0]], plain[pages[0]], rtol=2e-6, atol=0)
    assert (out[pages[2][0]] == -3).all()
    if T == 2:  # (all rows see a key of the other page)
        assert np.allclose(out[pages[2][1:]].double().sum(0).cpu().numpy(), 4.0, rtol=1e-5)


def table_case(B, P, Hkv, seed, hi, spare=3):
    rng = np.random.RandomState(seed)
    ctx = rng.randint(0, hi + 1, B)
    ctx[0] = hi
    if B > 2:
        ctx[1] = 0
    held = -(-ctx // P)
    num = int(held.sum()) + spare
    perm = rng.permutation(num)
    table = np.full((B, int(held.max()) + 2), -1)
    at = 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    w = (rng.rand(num, Hkv) ** 4).astype(np.float32)
    return ctx, table, num, w, rng


@pytest.mark.parametrize("B,P,Hkv,hi", [(1, 16, 1, 1), (1, 64, 4, 20000), (7, 16, 2, 900), (33, 48, 8, 4000), (300, 16, 3, 700), (1024, 32, 1, 300)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict(B, P, Hkv, hi, in_place):
    ctx, table, num, w, rng = table_case(B, P, Hkv, B + P, hi)
    for keep, sinks, recent in ((1, 0, 1), (3, 2, 1), (6, 1, 2), (40, 0, 5)):
        want, lens, freed = ref.evict(w, table, ctx, P, keep, sinks, recent)
        tb = i32(table)
        out = None if in_place else torch.full_like(tb, -9)
        new_ctx, count, status = i32([-5] * B), i32([-5]), i32([0])
        lst = i32([-7] * (len(freed) + 3))
        got = nk.evict_pages(P, torch.from_numpy(w).cuda(), tb, i32(ctx), keep, new_ctx, lst, count, sink_pages=sinks,
                             recent_pages=recent, out=out, status=status)
        assert np.array_equal(got.cpu().numpy(), want) and (got is tb) == in_place
        assert new_ctx.tolist() == lens and int(count.item()) == len(freed)
        assert lst.tolist() == freed + [-7] * 3 and int(status.item()) == 0
        if not in_place:
            assert np.array_equal(tb.cpu().numpy(), table)


@pytest.mark.parametrize("what", ["equal", "nearly_equal", "wide", "nan", "zeros"])
def test_evict_ties_and_ranges(what):
    ctx, table, num, w, rng = table_case(3, 16, 3, 9, 3000)
    if what == "equal":
        w[:] = np.float32([0.1, 0.2, 0.3])
        w[::3] = w[::3, ::-1]  # the same numbers in another order: the sums are exact, so equal
    elif what == "nearly_equal":
        w[:] = 1.0
        w[:, 1] += (rng.randint(0, 3, num) * 2.0 ** -23).astype(np.float32)
        w[:, 2] = (2.0 ** -40) * rng.randint(0, 5, num)
    elif what == "wide":
        w[:] = 2.0 ** rng.randint(-120, 100, w.shape)
        w[:, 1:] = w[:, :1]  # (sums of numbers further apart than 48 bits are rounded)
    elif what == "zeros":
        w[:] = 0
        w[::2] = -0.0
    for keep, sinks, recent in ((8, 1, 1), (100, 0, 3)):
        ws = w.copy()
        if what == "nan":
            ws[table[0, 20], 1] = np.nan
        plain = np.where(np.isnan(ws).any(1, keepdims=True), np.float32(-1e30), ws)
        want, lens, freed = ref.evict(plain, table, ctx, 16, keep, sinks, recent)
        tb, new_ctx, count, lst = i32(table), i32([0] * 3), i32([0]), i32([-7] * len(freed))
        nk.evict_pages(16, torch.from_numpy(ws).cuda(), tb, i32(ctx), keep, new_ctx, lst, count, sink_pages=sinks, recent_pages=recent)
        assert np.array_equal(tb.cpu().numpy(), want) and lst.tolist() == freed, (keep, sinks, recent)


def test_evict_nothing_and_the_widest_table():
    count, none, f = i32([-5]), i32([]), torch.zeros((4, 2), device="cuda")
    nk.evict_pages(16, f, i32(np.zeros((0, 4))), none, 3, none, i32([-7]), count)
    assert count.tolist() == [0]
    ctx, table, num, w, rng = table_case(1, 16, 2, 21, 16382 * 16 - 5)
    assert table.shape[1] == 16384
    want, lens, freed = ref.evict(w, table, ctx, 16, 900, 1, 2)
    tb, new_ctx, lst = i32(table), i32([0]), i32([-7] * len(freed))
    nk.evict_pages(16, torch.from_numpy(w).cuda(), tb, i32(ctx), 900, new_ctx, lst, count, sink_pages=1, recent_pages=2)
    assert np.array_equal(tb.cpu().numpy(), want) and lst.tolist() == freed and new_ctx.tolist() == lens


@pytest.mark.parametrize("T", [1, 16])
def test_captured_and_on_another_stream(T):
    c = make(("graph", 2, T, 24, 4, 256, 64, [3001, 900]))
    w = c.w
    want = torch.zeros((w.num_pages, w.Hkv), device="cuda")
    nk.page_weights(c.pool, c.q, c.bt, c.ctx, w.sm_scale, w.max_ctx, want)
    lists = [(torch.zeros_like(c.bt), i32([0] * w.B), i32([-7] * 50), i32([0])) for _ in range(3)]

    def step(mass, out, new_ctx, freed, count, **kw):
        nk.page_weights(c.pool, c.q, c.bt, c.ctx, w.sm_scale, w.max_ctx, mass, **kw)
        nk.evict_pages(w.P, mass, c.bt, c.ctx, 9, new_ctx, freed, count, out=out, **kw)

    mass = [torch.zeros_like(want) for _ in range(3)]
    step(mass[0], *lists[0])
    step(mass[2], *lists[2])  # (the kernels are loaded before the capture)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(mass[1], *lists[1])
    for _ in range(2):
        for t in (mass[1], *lists[1]):
            t.fill_(-7)
        g.replay()
        touched = want != 0
        assert torch.equal(mass[1][touched], want[touched])
        for x, y in zip(lists[0][:2] + lists[0][3:], lists[1][:2] + lists[1][3:]):
            assert torch.equal(x, y)
        assert torch.equal(lists[0][2], lists[1][2])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    step(mass[2], *lists[2], stream=st)
    st.synchronize()
    assert torch.equal(mass[2], want) and all(torch.equal(x, y) for x, y in zip(lists[0], lists[2]))


def test_evict_bad_data():
    ctx, table, num, w, rng = table_case(4, 16, 2, 4, 500)
    ctx[2], ctx[3] = -1, table.shape[1] * 16 + 1
    ok = ctx.copy()
    ok[2:] = 0
    want, lens, freed = ref.evict(w, table, ok, 16, 5, 1, 1)
    tb, out, new_ctx, count, status = i32(table), torch.full(table.shape, -9, dtype=torch.int32, device="cuda"), i32([-5] * 4), i32([0]), i32([0])
    lst = i32([-7] * (len(freed) - 2))
    nk.evict_pages(16, torch.from_numpy(w).cuda(), tb, i32(ctx), 5, new_ctx, lst, count, out=out, status=status)
    assert int(status.item()) == nk.NK_DEVFLAG_BAD_CTX | nk.NK_DEVFLAG_NO_PAGES and int(count.item()) == len(freed)
    got = out.cpu().numpy()
    assert np.array_equal(got[:2], want[:2]) and (got[2:] == -9).all()
    assert new_ctx.tolist() == lens[:2] + [0, 0] and lst.tolist() == freed[:-2]
    # a page outside the pool weighs nothing and is listed as -1
    ctx, table, num, w, rng = table_case(1, 16, 2, 5, 400)
    table[0, 7] = num
    wide = np.concatenate([w, np.zeros((1, 2), np.float32)])
    want, lens, freed = ref.evict(wide, table, ctx, 16, 6, 1, 1)
    lst, status = i32([-7] * len(freed)), i32([0])
    tb = i32(table)
    nk.evict_pages(16, torch.from_numpy(w).cuda(), tb, i32(ctx), 6, i32([0]), lst, i32([0]), status=status)
    assert int(status.item()) == nk.NK_DEVFLAG_BAD_PAGE
    assert lst.tolist() == [-1 if x == num else x for x in freed] and np.array_equal(tb.cpu().numpy(), want)


def test_steps_over_long_caches():
    """Prompts appended, their bounds made, evicted by the weights of their last tokens, then steps that append, select,
    attend and accumulate: the attention of every step against the plain form, and a full selection against the whole
    context's decode."""
    B, T, Hq, Hkv, D, P = 3, 4, 12, 2, 128, 16
    lens = [700, 333, 90]
    c = make(("steps", B, T, Hq, Hkv, D, P, lens), spare=40)
    w = c.w
    bounds = nk.PageBounds.empty(c.pool)
    nk.page_bounds(c.pool, bounds, c.bt, i32([0] * B), i32(np.cumsum([0] + lens)), status=c.status)
    mass = torch.full((w.num_pages, Hkv), 99.0, device="cuda")
    nk.page_weights(c.pool, c.q, c.bt, c.ctx, w.sm_scale, w.max_ctx, mass, status=c.status)
    keep = 12
    table, start, freed, count = c.bt.clone(), i32([0] * B), i32([-1] * 64), i32([0])
    want = ref.evict(mass.cpu().numpy(), c.bt_cpu.numpy(), lens, P, keep, 1, 2)
    nk.evict_pages(P, mass, table, c.ctx, keep, start, freed, count, sink_pages=1, recent_pages=2, status=c.status)
    assert np.array_equal(table.cpu().numpy(), want[0]) and start.tolist() == want[1]
    gen = torch.Generator(device="cuda").manual_seed(8)
    free = freed  # the pages that went serve the next steps
    for step in range(3):
        new = i32([T] * B)
        rows = B * T
        cu, ctx, slots, used = i32([0] * (B + 1)), i32([0] * B), torch.empty(rows, dtype=torch.int64, device="cuda"), i32([0])
        seen = start.clone()
        nk.step_tables(P, w.num_pages, start, new, free, table, cu, ctx, slots, used=used, status=c.status)
        free = free[int(used.item()):].contiguous()
        k, v = (torch.randn((rows, Hkv, D), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
        q = torch.randn((B, T, Hq, D), generator=gen, device="cuda").to(torch.bfloat16)
        nk.kv_append(c.pool, table, start, cu, k, v, status=c.status)
        nk.page_bounds(c.pool, bounds, table, start, cu, status=c.status)
        host, lengths = table.cpu(), ctx.tolist()
        top = max(lengths)
        lists = nk.page_select(bounds, q, table, ctx, P, top, 5, sink_pages=1, recent_pages=2, status=c.status)
        assert np.array_equal(lists.cpu().numpy(), ref.select(bounds.codes().cpu().numpy(), bounds.scales().cpu().numpy(),
                                                             q.double().cpu().numpy(), host.numpy(), lengths, P, 5, 1, 2))
        out = nk.paged_sparse_attn(c.pool, q, table, ctx, lists, w.sm_scale, top, status=c.status)
        compare(out, ref.sparse(c.pool.storage, w.num_pages, Hkv, P, D, host.numpy(), lengths, lists.cpu().numpy(), q, w.sm_scale), f"step {step}")
        full = nk.page_select(bounds, q, table, ctx, P, top, 40, status=c.status)
        compare(nk.paged_sparse_attn(c.pool, q, table, ctx, full, w.sm_scale, top),
                nk.paged_decode_attn(c.pool, q, table, ctx, w.sm_scale, top).double().cpu().numpy(), f"step {step}, all pages")
        before = mass.clone()
        prior = {(int(host[b, i]), h): float(before[int(host[b, i]), h]) for b in range(B) for i in range(-(-int(seen[b]) // P)) for h in range(Hkv)}
        nk.page_weights(c.pool, q, table, ctx, w.sm_scale, top, mass, prior=mass, seen=seen, status=c.status)
        check_weights(c, mass, ref.weights(c.pool.storage, w.num_pages, Hkv, P, D, host.numpy(), lengths, q, w.sm_scale), before, prior)
        # a verify round's end: the rows of refused drafts are given up
        p = torch.softmax(torch.randn((B, T, 50), generator=gen, device="cuda"), -1)
        d = torch.softmax(torch.randn((B, T - 1, 50), generator=gen, device="cuda"), -1)
        drafts = torch.multinomial(d.view(-1, 50), 1, generator=gen).view(B, T - 1).to(torch.int32)
        nxt = i32([0] * B)
        _, acc = nk.verify_drafts(p, d, drafts, torch.rand((B, T), generator=gen, device="cuda"), ctx_lens=ctx, next_start=nxt, status=c.status)
        assert nxt.tolist() == [L - T + 1 + a for L, a in zip(lengths, acc.tolist())]
        start = nxt
    assert int(c.status.item()) == 0
