"""nk_step_tables and nk_mrope on the GPU against plain 64-bit forms, and one
serving step (tables, rotary positions, append, attention) run together."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import quantized_paged_kv_cache_gb300 as nk

import _ref

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32), device="cuda")


def run_tables(P, num_pages, start, new, free, table, max_rows, with_pos=True, graph=False):
    B = len(start)
    t = dict(start=i32(start), new=i32(new), free=i32(free), table=i32(table), cu=i32([-5] * (B + 1)), ctx=i32([-5] * B),
             slots=torch.full((max_rows,), -7, dtype=torch.int64, device="cuda"),
             pos=i32([-7] * max_rows) if with_pos else None, used=i32([-5]), status=i32([0]))

    def call():
        nk.step_tables(P, num_pages, t["start"], t["new"], t["free"], t["table"], t["cu"], t["ctx"], t["slots"],
                       positions=t["pos"], used=t["used"], status=t["status"])

    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        g.replay()
        g.replay()
    else:
        call()
    torch.cuda.synchronize()
    return t


def make(B, P, seed, start_hi, new_hi, spare=3, slack=5):
    rng = np.random.RandomState(seed)
    start = rng.randint(0, start_hi + 1, B)
    new = rng.randint(0, new_hi + 1, B)
    held = -(-start // P)
    need = -(-(start + new) // P) - held
    num_pages = int(held.sum() + need.sum()) + spare
    perm = rng.permutation(num_pages)
    width = int((held + need).max()) + 2
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    return start.tolist(), new.tolist(), perm[at:], table, num_pages, int(new.sum()) + slack


def check_tables(t, want, with_pos=True):
    table, cu, ctx, slots, pos, used = want
    assert np.array_equal(t["table"].cpu().numpy(), table)
    assert np.array_equal(t["cu"].cpu().numpy(), cu)
    assert np.array_equal(t["ctx"].cpu().numpy(), ctx)
    assert np.array_equal(t["slots"].cpu().numpy(), slots)
    assert int(t["used"].item()) == used
    if with_pos:
        assert np.array_equal(t["pos"].cpu().numpy(), pos)


@pytest.mark.parametrize("B,P,start_hi,new_hi", [
    (1, 64, 0, 1), (1, 16, 1000, 1), (8, 64, 5000, 1), (3, 48, 100, 200), (33, 16, 70, 5), (257, 64, 300, 300),
    (1023, 32, 64, 40), (1024, 256, 600, 17), (5, 1, 7, 9)])
@pytest.mark.parametrize("graph", [False, True])
def test_tables(B, P, start_hi, new_hi, graph):
    start, new, free, table, pages, rows = make(B, P, 7 * B + P, start_hi, new_hi)
    if B == 1 and new_hi == 1:
        new, rows = [1], 6
    t = run_tables(P, pages, start, new, free, table, rows, graph=graph)
    want = _ref.tables(P, pages, start, new, free, table, rows, np.full(rows, -7), np.full(rows, -7))
    check_tables(t, want)
    assert int(t["status"].item()) == 0


def test_tables_without_positions_and_with_nothing_new():
    start, new, free, table, pages, rows = make(9, 16, 3, 60, 30)
    t = run_tables(16, pages, start, new, free, table, rows, with_pos=False)
    check_tables(t, _ref.tables(16, pages, start, new, free, table, rows, np.full(rows, -7), np.full(rows, -7)), False)
    t = run_tables(16, pages, start, [0] * 9, free, table, 4)
    check_tables(t, _ref.tables(16, pages, start, [0] * 9, free, table, 4, np.full(4, -7), np.full(4, -7)))
    assert int(t["used"].item()) == 0 and int(t["status"].item()) == 0


@pytest.mark.parametrize("graph", [False, True])
def test_tables_of_no_sequences(graph):
    t = run_tables(16, 8, [], [], [3, 1], np.zeros((0, 4)), 5, graph=graph)
    assert t["cu"].tolist() == [0] and int(t["used"].item()) == 0 and int(t["status"].item()) == 0
    assert t["slots"].tolist() == [-7] * 5 and t["pos"].tolist() == [-7] * 5  # rows behind the last stay


@pytest.mark.parametrize("case", ["negative_start", "negative_new", "past_table", "short_free", "no_free", "bad_free_page",
                                  "bad_held_page", "rows_past_buffer", "too_many_rows"])
def test_tables_bad_data_is_flagged(case):
    start, new, free, table, pages, rows = make(7, 16, 11, 60, 50)
    new[3], start[3] = 20, 21  # a partly filled page with new rows behind it
    held = -(-21 // 16)
    start2, new2, free2, table2, rows2 = list(start), list(new), free.copy(), table.copy(), sum(new) + 5
    table2[3, :held] = [0, 1][:held]
    width = table2.shape[1]
    flagged = nk.NK_DEVFLAG_BAD_POS
    if case == "negative_start":
        start2[2] = -1
    elif case == "negative_new":
        new2[2] = -4
    elif case == "past_table":
        new2[5] = width * 16 - start2[5] + 1
        rows2 = sum(new2) + 5
    elif case == "short_free":
        free2, flagged = free2[:3], nk.NK_DEVFLAG_NO_PAGES
    elif case == "no_free":
        free2, flagged = free2[:0], nk.NK_DEVFLAG_NO_PAGES
    elif case == "bad_free_page":
        free2[1], flagged = pages, nk.NK_DEVFLAG_BAD_PAGE
    elif case == "bad_held_page":
        table2[3, held - 1], flagged = -3, nk.NK_DEVFLAG_BAD_PAGE
    elif case == "rows_past_buffer":
        rows2 = sum(new2) - 6
    elif case == "too_many_rows":
        new2[1] = new2[4] = 2 ** 31 - 1
        t = run_tables(16, pages, start2, new2, free2, table2, rows2)
        assert int(t["status"].item()) & nk.NK_DEVFLAG_BAD_POS
        assert torch.all(t["slots"] == -7) and np.array_equal(t["table"].cpu().numpy(), table2)
        assert t["cu"].tolist()[5:] == [2 ** 31 - 1] * 3
        return
    want = _ref.tables(16, pages, start2, new2, free2, table2, rows2, np.full(rows2, -7), np.full(rows2, -7))
    t = run_tables(16, pages, start2, new2, free2, table2, rows2)
    check_tables(t, want)
    assert int(t["status"].item()) == flagged


# A bf16 result is off by its rounding (2^-8 of the value, half a step) and by what the fp32 rotation leaves: the angle
# (2^-23 turns from the frequency's double at position 2^31, 2^-25 from the fp32 fraction: together below 1e-6 radians,
# and 3e-7 of the reference's own 64-bit angle there) and sincospi and two fp32 roundings (3e-7), times |a| + |b|.
ROPE_ABS = 2.0 ** -19


def check_rope(got, x, pos, inv, sections, interleaved):
    want, size = _ref.mrope(x, pos, inv, sections, interleaved)
    err = (got.double() - want).abs()
    assert torch.all(err <= 2.0 ** -8 * want.abs() + ROPE_ABS * size), float((err - 2.0 ** -8 * want.abs()).max())
    rot = 2 * len(inv)
    assert torch.equal(got[..., rot:], x[..., rot:])


def rope_case(rows, Hq, Hkv, D, sections, far, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn((rows, Hq + 2 * Hkv, D), generator=g, device="cuda").bfloat16()
    pos = torch.randint(0, far, (len(sections), rows), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    half = sum(sections)
    inv = 1e6 ** (-torch.arange(half, dtype=torch.float64) / half)
    return qkv, pos, inv


@pytest.mark.parametrize("rows,Hq,Hkv,D,sections,interleaved,far", [
    (1, 24, 4, 256, (32, 48, 48), False, 1000),
    (8, 24, 4, 256, (32, 48, 48), False, 262144),
    (37, 16, 2, 128, (12, 10, 10), True, 262144),
    (1000, 8, 8, 64, (32,), False, 2 ** 31 - 1),
    (5, 3, 1, 64, (0, 8, 0), False, 5000),
    (9, 2, 1, 256, (100, 10, 10, 8), True, 100000),
    (2049, 5, 5, 128, (24, 20, 20), True, 100000),
    (6, 7, 3, 40, (8,), False, 64),
    (4, 24, 0, 256, (128,), False, 64),
])
def test_mrope(rows, Hq, Hkv, D, sections, interleaved, far):
    qkv, pos, inv = rope_case(rows, Hq, Hkv, D, sections, far, rows)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
    before = qkv.clone()
    qo, ko = nk.mrope(q, k, pos, inv, sections, interleaved=interleaved)
    torch.cuda.synchronize()
    assert torch.equal(qkv, before)
    check_rope(qo, q, pos, inv, sections, interleaved)
    if Hkv:
        check_rope(ko, k, pos, inv, sections, interleaved)
    # in place, inside the fused rows: the same values, and the value rows untouched
    nk.mrope(q, k, pos, inv, sections, interleaved=interleaved, q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(qkv[:, Hq + Hkv:], before[:, Hq + Hkv:])


def test_mrope_negative_positions_and_non_finite_rows():
    qkv, pos, inv = rope_case(12, 2, 1, 64, (16, 8, 8), 1000, 5)
    pos[0, ::2] = -pos[0, ::2] - 2 ** 30
    q, k = qkv[:, :2], qkv[:, 2:3]
    qo, _ = nk.mrope(q, k, pos, inv, (16, 8, 8))
    check_rope(qo, q, pos, inv, (16, 8, 8), False)
    q[3, 1, 5] = float("nan")
    q[4, 0, 9] = float("inf")
    qo2, _ = nk.mrope(q, k, pos, inv, (16, 8, 8))
    bad = torch.zeros_like(qo, dtype=torch.bool)
    bad[3, 1, [5, 37]] = True
    bad[4, 0, [9, 41]] = True
    assert torch.equal(qo2[~bad], qo[~bad]) and not torch.isfinite(qo2[bad]).any()


def test_mrope_rows_behind_the_last_stay_and_graphs_replay():
    qkv, pos, inv = rope_case(40, 4, 2, 128, (24, 20, 20), 9000, 6)
    q, k = qkv[:, :4], qkv[:, 4:6]
    n = i32([40])
    full_q, full_k = nk.mrope(q, k, pos, inv, (24, 20, 20))
    qo, ko = torch.full_like(full_q, 7.0), torch.full_like(full_k, 7.0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nk.mrope(q, k, pos, inv, (24, 20, 20), q_out=qo, k_out=ko, num_rows=n)
    for rows in (0, 1, 23, 40, 1000):
        qo.fill_(7.0), ko.fill_(7.0), n.fill_(rows)
        g.replay()
        torch.cuda.synchronize()
        m = min(rows, 40)
        assert torch.equal(qo[:m], full_q[:m]) and torch.equal(ko[:m], full_k[:m])
        assert torch.all(qo[m:] == 7.0) and torch.all(ko[m:] == 7.0)


@pytest.mark.parametrize("D,Hq,Hkv,P,window,sinks", [(256, 24, 4, 64, 0, 0), (128, 16, 2, 16, 100, 5)])
def test_a_step_of_continuous_batching(D, Hq, Hkv, P, window, sinks):
    """Three steps of a serving loop as a user writes them: tables and slot map, rotary positions, append, attention of the
    step's ragged tokens, on one stream without a host synchronisation; against the 64-bit forms at the end of each step."""
    rng = np.random.RandomState(5)
    B, width, pages = 5, 24 * 64 // P, 140 * 64 // P
    perm = rng.permutation(pages)
    table, lens = i32(np.full((B, width), -1)), np.zeros(B, dtype=int)
    pool = nk.KVPool.empty(pages, P, Hkv, D, fill=0xFF)
    status = i32([0])
    inv = 1e6 ** (-torch.arange(D // 4, dtype=torch.float64) * 4 / D)
    sections = (D // 4 - 2 * (D // 12), D // 12, D // 12)
    g = torch.Generator(device="cuda").manual_seed(9)
    keys = [torch.empty((0, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(B)]
    taken = 0
    for step_new in ([300, 0, 77, 1, 500], [1, 40, 1, 1, 1], [4, 4, 200, 0, 1]):
        start, new = lens.copy(), np.asarray(step_new)
        total, rows = int(new.sum()), int(new.sum()) + 9  # buffers for the largest step
        free = i32(perm[taken:])
        cu, ctx = i32([0] * (B + 1)), i32([0] * B)
        slots, pos, used = torch.full((rows,), -7, dtype=torch.int64, device="cuda"), i32([0] * rows), i32([0])
        qkv = torch.randn((rows, Hq + 2 * Hkv, D), generator=g, device="cuda").bfloat16()
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        startd, newd = i32(start), i32(new)
        nk.step_tables(P, pages, startd, newd, free, table, cu, ctx, slots, positions=pos, used=used, status=status)
        axes = torch.stack([pos, pos // 7, pos % 7]).contiguous()
        qr, kr = nk.mrope(q, k, axes, inv, sections, interleaved=True, num_rows=cu[B:])
        nk.kv_append(pool, table, startd, cu, kr[:total].contiguous(), v[:total].contiguous(), status=status)
        out = nk.paged_chunk_attn(pool, qr, cu, table, ctx, 1 / D ** 0.5, width * P, window=window, sinks=sinks, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        taken += int(used.item())
        lens = start + new
        assert ctx.tolist() == lens.tolist() and cu.tolist() == [0] + np.cumsum(new).tolist()
        # the slots are where the rows went
        K, _ = _ref.dequantized(pool.storage, pages, Hkv, P, D)
        flat = K.transpose(1, 2).reshape(pages * P, Hkv, D)[slots[:total]]
        scale = kr[:total].double().unflatten(-1, (D // 64, 64)).abs().amax(-1, keepdim=True) / 127
        # a code is off by half a step, of 127 (and the scale by its own rounding, below 2^-23 of the value)
        assert torch.all((flat.unflatten(-1, (D // 64, 64)) - kr[:total].double().unflatten(-1, (D // 64, 64))).abs() <= scale * 0.5001)
        check_rope(qr[:total], q[:total], axes[:, :total], inv, sections, True)
        want = _ref.attention(pool.storage, pages, Hkv, P, D, table, lens.tolist(), new.tolist(), qr[:total], 1 / D ** 0.5, window, sinks)
        # the chunk attention's tolerance: half a bf16 step and 4e-3 for its fp16 operands (tests/test_gpu_chunk.py)
        err = (out[:total].double() - want).abs()
        assert torch.all(err <= 2.0 ** -8 * want.abs() + 4e-3)
        # a decoding batch: the same tokens through the windowed decode
        if (new == new[0]).all():
            continue
        one = [b for b in range(B) if lens[b] > 0]
        qd = qr[:len(one)].reshape(len(one), 1, Hq, D).contiguous()
        args = (pool, qd, table[one].contiguous(), ctx[one].contiguous(), 1 / D ** 0.5, width * P)
        got = nk.paged_window_attn(*args, window, sinks=sinks) if window else nk.paged_decode_attn(*args)
        want = _ref.attention(pool.storage, pages, Hkv, P, D, table[one], lens[one].tolist(), [1] * len(one), qd, 1 / D ** 0.5,
                              window, sinks).reshape(got.shape)
        assert torch.all((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 4e-3)


def test_step_operators_follow_the_stream_order():
    """A side stream holds the whole step; the calls read what kernels before them on that stream wrote."""
    P, D, Hq, Hkv, B = 16, 128, 8, 2, 3
    pool = nk.KVPool.empty(64, P, Hkv, D, fill=0)
    side = torch.cuda.Stream()
    outs = []
    for rep in range(2):
        g = torch.Generator(device="cuda").manual_seed(3)
        qkv = torch.randn((60, Hq + 2 * Hkv, D), generator=g, device="cuda").bfloat16()
        src = i32([30, 1, 29])
        torch.cuda.synchronize()
        stream = side if rep else torch.cuda.current_stream()
        with torch.cuda.stream(stream):
            if rep:
                torch.cuda._sleep(20_000_000)  # everything below is enqueued long before it runs
            start, new = torch.zeros(B, dtype=torch.int32, device="cuda"), src * 1
            table = torch.full((B, 8), -1, dtype=torch.int32, device="cuda")
            free = torch.arange(63, -1, -1, dtype=torch.int32, device="cuda")
            cu, ctx = torch.zeros(B + 1, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
            slots, pos = torch.zeros(60, dtype=torch.int64, device="cuda"), torch.zeros(60, dtype=torch.int32, device="cuda")
            nk.step_tables(P, 64, start, new, free, table, cu, ctx, slots, positions=pos)
            q, k = nk.mrope(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], pos[None].contiguous(), torch.ones(64, dtype=torch.float64), (64,))
            nk.kv_append(pool, table, start, cu, k, qkv[:, Hq + Hkv:].contiguous())
            outs.append(nk.paged_chunk_attn(pool, q, cu, table, ctx, 0.1, 128))
        stream.synchronize()
    assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("raw", [False, True])
def test_memory_of_a_call_belongs_to_its_stream(raw, monkeypatch):
    pool = nk.KVPool.empty(4, 16, 1, 64, fill=0)
    q, k = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, 1, 64, dtype=torch.bfloat16, device="cuda")
    table, ctx, cu = i32([[0, 1]]), i32([20]), i32([0, 3])
    pos, inv = i32([[0, 1, 2]]), torch.ones(32, dtype=torch.float64)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    arg, seen, empty = side.cuda_stream if raw else side, [], torch.empty

    def watched(*a, **kw):
        if "cuda" in str(kw.get("device", "")):
            seen.append(torch.cuda.current_stream().cuda_stream)
        return empty(*a, **kw)

    monkeypatch.setattr(torch, "empty", watched)
    nk.mrope(q, k, pos, inv, (32,), stream=arg)
    nk.paged_window_attn(pool, q[:1].view(1, 1, 2, 64), table, ctx, 0.1, 32, 8, stream=arg)
    nk.paged_chunk_attn(pool, q, cu, table, ctx, 0.1, 32, stream=arg)
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert len(seen) == 6 and set(seen) == {side.cuda_stream}


def test_tensors_of_another_device_are_refused(monkeypatch):
    pool = nk.KVPool.empty(4, 16, 1, 64, fill=0)
    x, y = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, 1, 64, dtype=torch.bfloat16, device="cuda")
    table, ctx, cu, z, slots = i32([[0, 1]]), i32([20]), i32([0, 3]), i32([0]), torch.zeros(4, dtype=torch.int64, device="cuda")
    monkeypatch.setattr(nk, "_here", lambda: torch.cuda.current_device() + 1)  # as if that one were current
    for call in (lambda: nk.step_tables(16, 4, z, z, z, table, cu, ctx, slots),
                 lambda: nk.mrope(x, y, i32([[0, 1, 2]]), torch.ones(32, dtype=torch.float64), (32,)),
                 lambda: nk.paged_window_attn(pool, x[:1].view(1, 1, 2, 64), table, ctx, 0.1, 32, 8),
                 lambda: nk.paged_chunk_attn(pool, x, cu, table, ctx, 0.1, 32)):
        with pytest.raises(ValueError, match="current device"):
            call()


def test_arguments_past_32_bits():
    pool = nk.KVPool.empty(4, 16, 1, 64, fill=0)
    x = torch.randn(3, 2, 64, device="cuda").bfloat16()
    v = torch.randn(20, 1, 64, device="cuda").bfloat16()
    table, ctx, cu = i32([[0, 1]]), i32([20]), i32([0, 3])
    nk.kv_append(pool, table, i32([0]), i32([0, 20]), v, v)
    whole = nk.paged_chunk_attn(pool, x, cu, table, ctx, 0.1, 32)
    assert torch.equal(nk.paged_chunk_attn(pool, x, cu, table, ctx, 0.1, 32, window=2**32 + 3), whole)
    assert torch.equal(nk.paged_chunk_attn(pool, x, cu, table, ctx, 0.1, 32, window=1, sinks=2**32), whole)
    q = x.view(1, 3, 2, 64)
    all_keys = nk.paged_decode_attn(pool, q, table, ctx, 0.1, 32)
    assert torch.equal(nk.paged_window_attn(pool, q, table, ctx, 0.1, 32, 2**32 + 3), all_keys)
    for attn in (lambda m: nk.paged_chunk_attn(pool, x, cu, table, ctx, 0.1, m),
                 lambda m: nk.paged_window_attn(pool, q, table, ctx, 0.1, m, 8)):
        with pytest.raises(ValueError):
            attn(2**32 + 32)
    pos, inv = i32([[0, 1, 2]]), torch.ones(32, dtype=torch.float64)
    with pytest.raises(ValueError):  # no row count in it
        nk.mrope(x, x[:, :1], pos, inv, (32,), num_rows=cu[2:])


def test_first_call_of_a_process_may_be_captured():
    """Kernels whose code is not loaded yet, in a graph capture."""
    code = """
import torch, quantized_paged_kv_cache_gb300 as nk
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
for D, P, Hq in ((256, 64, 24), (64, 16, 4)):
    pool = nk.KVPool.empty(4, P, 2, D, fill=0)
    x = torch.ones(3, Hq, D, dtype=torch.bfloat16, device="cuda")
    start, new, free, table = i32([5]), i32([3]), i32([1, 2]), i32([[0, -1]])
    cu, ctx, slots = i32([0, 0]), i32([0]), torch.zeros(3, dtype=torch.int64, device="cuda")
    pos, inv = i32([[5, 6, 7]]), torch.ones(32, dtype=torch.float64)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nk.step_tables(P, 4, start, new, free, table, cu, ctx, slots)
        q, k = nk.mrope(x, x[:, :2], pos, inv, (32,))
        nk.kv_append(pool, table, start, cu, k, k)
        a = nk.paged_chunk_attn(pool, q, cu, table, ctx, 0.1, 2 * P, window=8)
        b = nk.paged_window_attn(pool, q.view(1, 3, Hq, D), table, ctx, 0.1, 2 * P, 8)
    g.replay()
    torch.cuda.synchronize()
    assert (a.float() - b.view_as(a).float()).abs().max().item() < 2e-2 and a.float().abs().max().item() > 0.5
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root, timeout=300)


def test_two_graphs_with_workspaces_of_their_own_run_at_once():
    rng = np.random.RandomState(8)
    D, P, Hq, Hkv = 128, 16, 16, 2
    calls = []
    for i in range(2):
        L = [int(x) for x in rng.randint(200, 3000, 6)]
        pages = [-(-n // P) for n in L]
        pool = nk.KVPool.empty(sum(pages), P, Hkv, D, fill=0)
        table = np.full((6, max(pages)), -1)
        at = 0
        for b, n in enumerate(pages):
            table[b, :n] = np.arange(at, at + n)
            at += n
        table = i32(table)
        rows = sum(L)
        k, v = (torch.randn(rows, Hkv, D, device="cuda").bfloat16() for _ in range(2))
        nk.kv_append(pool, table, i32([0] * 6), i32(np.concatenate(([0], np.cumsum(L)))), k, v)
        new = [1, 40, 3, 0, 17, 150]
        q = torch.randn(sum(new), Hq, D, device="cuda").bfloat16()
        cu, ctx = i32(np.concatenate(([0], np.cumsum(new)))), i32(L)
        qd = torch.randn(6, 2, Hq, D, device="cuda").bfloat16()
        ws = [torch.empty(nk.chunk_workspace_bytes(D), dtype=torch.uint8, device="cuda"),
              torch.empty(nk.decode_workspace_bytes(6, 2, Hq, Hkv, D), dtype=torch.uint8, device="cuda")]
        out = [torch.zeros_like(q), torch.zeros_like(qd)]

        def call(pool=pool, table=table, q=q, cu=cu, ctx=ctx, qd=qd, ws=ws, out=out, top=max(L)):
            nk.paged_chunk_attn(pool, q, cu, table, ctx, 0.1, top, window=500, sinks=3, workspace=ws[0], out=out[0])
            nk.paged_window_attn(pool, qd, table, ctx, 0.1, top, 150, 5, workspace=ws[1], out=out[1])

        call()
        torch.cuda.synchronize()
        want = [o.clone() for o in out]
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g, stream=s):
            call()
        calls.append((g, s, out, want, call))  # (call holds the tensors that the graph works on)
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s, out, want, _ in calls:
            with torch.cuda.stream(s):
                for o in out:
                    o.zero_()
                for _ in range(4):
                    g.replay()
        torch.cuda.synchronize()
        for g, s, out, want, _ in calls:
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_slots_and_rows_past_32_bits():
    # the last pages of a pool of 2^33 slots
    pages = 2**27
    t = run_tables(64, pages, [130, 0], [70, 65], [pages - 1, 3, pages - 2], [[5, 6, pages - 3, -1], [-1] * 4], 135)
    want = [(pages - 3) * 64 + 2 + i for i in range(62)] + [(pages - 1) * 64 + i for i in range(8)]
    want += [3 * 64 + i for i in range(64)] + [(pages - 2) * 64]
    assert t["slots"].tolist() == want and int(t["status"].item()) == 0
    # rows of a buffer further apart than 2^31 elements in all
    stride, Hq, D = 2**30, 3, 64
    buf = torch.empty(2 * stride + 4 * D, dtype=torch.bfloat16, device="cuda")
    q, k = buf.as_strided((3, Hq, D), (stride, D, 1)), buf.as_strided((3, 1, D), (stride, D, 1), Hq * D)
    x, y = torch.randn(3, Hq, D, device="cuda").bfloat16(), torch.randn(3, 1, D, device="cuda").bfloat16()
    q.copy_(x), k.copy_(y)
    pos, inv = i32([[1, 50, 9000]]), 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)
    want = nk.mrope(x, y, pos, inv, (32,))
    nk.mrope(q, k, pos, inv, (32,), q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_negative_numbers_past_32_bits_are_refused():
    """They must not come out as small positive ones on the way into the C calls."""
    D, P, i32 = 64, 16, torch.int32
    pool = nk.KVPool.empty(2, P, 2, D, fill=0)
    table = torch.zeros(1, 2, dtype=i32, device="cuda")
    ctx, cu = torch.tensor([1], dtype=i32, device="cuda"), torch.tensor([0, 1], dtype=i32, device="cuda")
    x = torch.randn(1, 2, D, device="cuda").bfloat16()
    for window, sinks in ((5 - 2**32, 0), (5, 5 - 2**32), (-5, 0), (5, -5)):
        with pytest.raises(nk.NKError):
            nk.paged_window_attn(pool, x.unsqueeze(0), table, ctx, 0.1, 32, window, sinks=sinks)
        with pytest.raises(nk.NKError):
            nk.paged_chunk_attn(pool, x, cu, table, ctx, 0.1, 32, window=window, sinks=sinks)
    with pytest.raises(ValueError):
        nk.paged_window_attn(pool, x.unsqueeze(0), table, ctx, 0.1, 32 - 2**32, 5)
    with pytest.raises(ValueError):
        nk.paged_chunk_attn(pool, x, cu, table, ctx, 0.1, 32 - 2**32, window=5)
    slots = torch.zeros(4, dtype=torch.int64, device="cuda")
    for page_size, pages in ((2**32 + 16, 2), (16, 2**32 + 2), (16 - 2**32, 2), (16, 2 - 2**32)):
        with pytest.raises(ValueError):
            nk.step_tables(page_size, pages, ctx, ctx, ctx, table, cu, ctx.clone(), slots)
