"""Decode / verify attention over a sliding window with sinks
(nk_paged_window_attn) against the plain 64-bit form."""
import pytest
import torch

import quantized_paged_kv_cache_gb300 as nk
from quantized_paged_kv_cache_gb300 import workloads as wl

import _ref
from _cases import build, compare

pytestmark = pytest.mark.gpu

SHAPES = [
    # name, B, T, Hq, Hkv, D, P, ctx_lens
    ("t1_d256", 3, 1, 24, 4, 256, 64, [1, 700, 4099]),
    ("t4_d256", 2, 4, 24, 4, 256, 64, [4, 3001]),
    ("t16_d256", 2, 16, 24, 4, 256, 64, [16, 1500]),      # column chunks
    ("t1_d128_p16", 5, 1, 16, 2, 128, 16, [1, 15, 16, 17, 900]),
    ("t3_d64_p32", 2, 3, 8, 8, 64, 32, [1000, 50]),
    ("t2_d128_p128", 2, 2, 6, 2, 128, 128, [1300, 129]),
    ("t5_d64_p48", 3, 5, 10, 2, 64, 48, [5, 500, 49]),
]
WINDOWS = [(1, 0), (1, 3), (16, 0), (64, 4), (100, 5), (129, 130), (500, 64), (700, 1 << 20), (1 << 30, 0)]


def reference(c, window, sinks):
    w = c.w
    return _ref.attention(c.pool.storage, w.num_pages, w.Hkv, w.P, w.D, c.bt, w.ctx_lens, [w.T] * w.B, c.q, w.sm_scale,
                          window, sinks).cpu().numpy()


def call(c, window, sinks, **kw):
    w = c.w
    return nk.paged_window_attn(c.pool, c.q, kw.pop("bt", c.bt), kw.pop("ctx", c.ctx), w.sm_scale, w.max_ctx, window,
                                sinks=sinks, **kw)


@pytest.mark.parametrize("shape", SHAPES, ids=[s[0] for s in SHAPES])
def test_window_matches_reference(shape):
    name, B, T, Hq, Hkv, D, P, lens = shape
    w = wl.custom(name, B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, P=P, ctx_lens=lens, seed=91,
                  num_pages=sum((L + P - 1) // P for L in lens) + 2, outlier_channels=2, outlier_scale=8.0)
    c = build(w, fill=0xFF, oracle_pool=False)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for window, sinks in WINDOWS:
        ref = reference(c, window, sinks)
        for n in (0, 1, 7):
            out = call(c, window, sinks, num_ctas=n, status=status)
            compare(out, ref, f"{name} window={window} sinks={sinks} ctas={n}")
        assert torch.equal(out, call(c, window, sinks, num_ctas=7)), "run-to-run results differ"
    assert int(status.item()) == 0


@pytest.mark.parametrize("B,T", [(64, 1), (70, 2), (33, 1), (32, 2), (300, 1)])
def test_a_batch_of_windows_split_evenly_over_its_units(B, T):
    lens = [150 + 37 * b % 260 for b in range(B)]
    lens[1], lens[B // 2] = T, 60  # (most units have the window's pages, some fewer)
    w = wl.custom(f"even{B}", B=B, T=T, Hq=16, Hkv=2, D=128, P=16, ctx_lens=lens, seed=94,
                  num_pages=sum((L + 15) // 16 for L in lens) + 2, outlier_channels=2, outlier_scale=8.0)
    c = build(w, fill=0xFF, oracle_pool=False)
    for window, sinks in ((100, 5), (40, 0)):
        compare(call(c, window, sinks), reference(c, window, sinks), f"{B} sequences, window {window}")


def test_a_window_over_everything_is_the_whole_context():
    w = wl.custom("win_all", B=2, T=4, Hq=24, Hkv=4, D=256, P=64, ctx_lens=[900, 333], seed=92)
    c = build(w, oracle_pool=False)
    want = nk.paged_decode_attn(c.pool, c.q, c.bt, c.ctx, w.sm_scale, w.max_ctx)
    assert torch.equal(call(c, w.max_ctx, 0), want)
    compare(call(c, w.max_ctx - 1, 1), want.double().cpu().numpy(), "one key short of everything, which is a sink")


@pytest.mark.parametrize("T", [1, 4])
def test_pages_between_sinks_and_window_are_not_read(T):
    w = wl.custom("win_freed", B=2, T=T, Hq=24, Hkv=4, D=256, P=64, ctx_lens=[2000, 1111], seed=93, num_pages=60)
    c = build(w, oracle_pool=False)
    window, sinks = 200, 70
    want = call(c, window, sinks)
    bt = c.bt.clone()
    for b, L in enumerate(w.ctx_lens):
        bt[b, 2:(L - T - window + 1) // 64] = -1  # given back: the sinks take two pages
        bt[b, -(-L // 64):] = 1 << 30
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = call(c, window, sinks, bt=bt, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and torch.equal(out, want)


def test_scaled_inputs_and_bad_contexts():
    for which, s in (("q", -12), ("v", -12), ("v", 10)):
        w = wl.custom(f"win_{which}{s}", B=1, T=2, Hq=24, Hkv=4, D=256, P=64, ctx_lens=[1500], seed=94,
                      **{f"{which}_scale": 2.0 ** s})
        c = build(w, oracle_pool=False)
        back = 2.0 ** -s if which == "v" else 1.0
        compare(call(c, 333, 5).double() * back, reference(c, 333, 5) * back, w.name)
    w = wl.custom("win_bad", B=3, T=2, Hq=8, Hkv=2, D=128, P=16, ctx_lens=[64, 300, 200], seed=95)
    c = build(w, oracle_pool=False)
    ref = reference(c, 40, 2)
    ctx = c.ctx.clone()
    ctx[0], ctx[2] = 1, w.max_ctx + 1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = call(c, 40, 2, ctx=ctx, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) & nk.NK_DEVFLAG_BAD_CTX
    compare(out[1], ref[2:4], "valid sequence between bad ones")


def test_window_replays_in_a_graph_on_a_side_stream():
    w = wl.custom("win_graph", B=4, T=1, Hq=16, Hkv=2, D=128, P=16, ctx_lens=[900, 10, 333, 64], seed=96)
    c = build(w, oracle_pool=False)
    want = call(c, 100, 4)
    ws = torch.empty(nk.decode_workspace_bytes(w.B, w.T, w.Hq, w.Hkv, w.D), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        call(c, 100, 4, workspace=ws, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("D,P,T", [(256, 64, 1), (256, 64, 4), (128, 16, 2)])
def test_the_last_positions_that_32_bits_hold(D, P, T):
    """A context of 2^31 - 1 tokens (its pages far from the window were given back) is the one of 2,047 tokens."""
    Hq, Hkv, near, far = 24, 4, 2047, 2**31 - 1
    shift = (far - near) // P
    pool = nk.KVPool.empty(2048 // P, P, Hkv, D, fill=0)
    table = torch.randperm(2048 // P, device="cuda").int().view(1, -1)
    k, v = (torch.randn(near, Hkv, D, device="cuda").bfloat16() for _ in range(2))
    lens = [torch.tensor([n], dtype=torch.int32, device="cuda") for n in (near, far, 0)]
    cu = torch.tensor([0, near], dtype=torch.int32, device="cuda")
    nk.kv_append(pool, table, lens[2], cu, k, v)
    long = torch.full((1, shift + 2048 // P), -1, dtype=torch.int32, device="cuda")
    long[:, shift:] = table
    q = torch.randn(1, T, Hq, D, device="cuda").bfloat16()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for window in (1, 100, 1500):
        a = nk.paged_window_attn(pool, q, table, lens[0], 0.1, near, window, status=status)
        b = nk.paged_window_attn(pool, q, long, lens[1], 0.1, far, window, status=status)
        assert torch.equal(a, b), f"window {window}"
        rows = torch.randn(70, Hq, D, device="cuda").bfloat16()
        cu = torch.tensor([0, 70], dtype=torch.int32, device="cuda")
        a = nk.paged_chunk_attn(pool, rows, cu, table, lens[0], 0.1, near, window=window, status=status)
        b = nk.paged_chunk_attn(pool, rows, cu, long, lens[1], 0.1, far, window=window, status=status)
        assert torch.equal(a, b), f"chunk, window {window}"
    assert int(status.item()) == 0


@pytest.mark.parametrize("D,P", [(256, 64), (128, 16)])
def test_pages_and_rows_past_4_gib(D, P):
    """Pages at the end of a pool of more than 2^32 bytes, query rows past 2^32 bytes."""
    Hq, Hkv, n = 24, 4, 1000
    used = -(-n // P)
    big_pages = 2**32 // (nk.kv_chunk_bytes(P, D) * Hkv) + used + 1
    k, v = (torch.randn(n, Hkv, D, device="cuda").bfloat16() for _ in range(2))
    start, cu, ctx = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0], [0, n], [n]))
    at = torch.arange(used, dtype=torch.int32, device="cuda").view(1, -1)
    pools = [(nk.KVPool.empty(used, P, Hkv, D), at), (nk.KVPool.empty(big_pages, P, Hkv, D), at + (big_pages - used))]
    base = 2**32 // (Hq * D * 2) + 1
    q = torch.randn(33, Hq, D, device="cuda").bfloat16()
    far, out = (torch.empty(base + 33, Hq, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    far[base:] = q
    got = []
    for pool, table in pools:
        nk.kv_append(pool, table, start, cu, k, v)
        for window in (300, n):
            got.append(nk.paged_window_attn(pool, q[:2].unsqueeze(0), table, ctx, 0.1, n, window))
            got.append(nk.paged_chunk_attn(pool, q, torch.tensor([0, 33], dtype=torch.int32, device="cuda"), table, ctx, 0.1, n,
                                           window=window))
            nk.paged_chunk_attn(pool, far, torch.tensor([base, base + 33], dtype=torch.int32, device="cuda"), table, ctx, 0.1,
                                n, window=window, out=out)
            assert torch.equal(out[base:], got[-1])
    assert all(torch.equal(a, b) for a, b in zip(got[:4], got[4:]))
