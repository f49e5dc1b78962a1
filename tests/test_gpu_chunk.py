"""Attention of ragged chunks over the paged INT8 cache (nk_paged_chunk_attn)
against the plain 64-bit form.

Tolerance. The output's bf16 rounding is off by at most 2^-8 of the value
(half a step; 1.65e-3 of the norm over many values). Before it, K and V enter
the products as fp16(code * fp16(scale)) and P as fp16: roundings of at most
2^-11 of each factor, 2^-11 / sqrt(3) in the mean square. A score is then off
by sm_scale |q k| 2^-11 sqrt(2/3) = 4e-4 for rows of N(0, 1), plus the scale's
rounding, 2.8e-4 of the score's group parts (scores of some units: up to about
1e-3), and O moves by sum_n p_n ds_n (v_n - O): at most six times
sqrt(sum p^2) 5e-4 |v - O|, 4e-3 for V rows of N(0, 1) when a few keys hold all
the weight. So: every element within 2^-8 |O| + 4e-3, and the norm of the
difference within sqrt(1.65^2 + 3 * 0.9^2) e-3 = 2.3e-3 of the norm, taken as
2.5e-3."""
import numpy as np
import pytest
import torch

import quantized_paged_kv_cache_gb300 as nk
from quantized_paged_kv_cache_gb300 import workloads as wl

import _ref
from _cases import build

pytestmark = pytest.mark.gpu


class Chunk:
    def __init__(self, name, qlens, ctx, Hq, Hkv, D, P, seed=71, fill=0xFF, **kw):
        self.w = wl.custom(name, B=len(ctx), T=1, Hq=Hq, Hkv=Hkv, D=D, P=P, ctx_lens=ctx, seed=seed,
                           num_pages=sum(-(-L // P) for L in ctx) + 2, **kw)
        self.c = build(self.w, fill=fill, oracle_pool=False)
        self.qlens = list(qlens)
        g = torch.Generator(device="cuda").manual_seed(seed)
        total = sum(qlens)
        self.q = (torch.randn((total, Hq, D), generator=g, device="cuda") * self.w.q_scale).bfloat16()
        self.cu = torch.tensor([0] + np.cumsum(qlens).tolist(), dtype=torch.int32, device="cuda")

    def run(self, window=0, sinks=0, **kw):
        return nk.paged_chunk_attn(self.c.pool, kw.pop("q", self.q), kw.pop("cu", self.cu), kw.pop("bt", self.c.bt),
                                   kw.pop("ctx", self.c.ctx), self.w.sm_scale, self.w.max_ctx, window=window, sinks=sinks,
                                   **kw)

    def ref(self, window=0, sinks=0):
        w = self.w
        return _ref.attention(self.c.pool.storage, w.num_pages, w.Hkv, w.P, w.D, self.c.bt, w.ctx_lens, self.qlens,
                              self.q, w.sm_scale, window, sinks)


def check(out, ref, what="", unit=1.0, roundings=1):
    """`roundings`: 2 where ref is itself a bf16 result. Two values that round to neighbours may be arbitrarily close, so
    the two results may lie a whole step, two halves of at most 2^-8 of the value, apart."""
    got, ref = out.double() / unit, ref / unit
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    err = (got - ref).abs()
    worst = float((err - roundings * 2.0 ** -8 * ref.abs()).max())
    rel = float((got - ref).norm() / ref.norm().clamp(min=1e-300))
    assert worst <= 4e-3 and rel <= 2.5e-3, f"{what}: {worst:.3e} past half a step, relative norm {rel:.3e}"


SHAPES = [
    # name, query tokens, contexts, Hq, Hkv, D, P
    ("one_token", [1], [1], 24, 4, 256, 64),
    ("one_block", [7], [40], 8, 2, 256, 64),
    ("first_chunk", [200], [200], 24, 4, 256, 64),
    ("after_history", [64, 33], [700, 4099], 24, 4, 256, 64),
    ("ragged", [1, 0, 130, 5, 1, 77], [900, 64, 130, 2000, 1, 1500], 16, 2, 128, 16),
    ("mixed_d256", [1, 300, 1, 1], [3000, 1000, 64, 65], 24, 4, 256, 64),
    ("g1_d64", [50, 129, 128], [300, 129, 1000], 8, 8, 64, 32),
    ("p48", [90, 3], [500, 49], 10, 2, 64, 48),
    ("p256", [40, 260], [900, 260], 6, 2, 128, 256),
    ("p16_d256", [37, 2], [999, 17], 14, 2, 256, 16),
    ("long", [130], [20000], 16, 2, 128, 64),
]


@pytest.mark.parametrize("shape", SHAPES, ids=[s[0] for s in SHAPES])
def test_chunk_matches_reference(shape):
    name, qlens, ctx, Hq, Hkv, D, P = shape
    k = Chunk(name, qlens, ctx, Hq, Hkv, D, P, outlier_channels=2, outlier_scale=8.0)
    ref = k.ref()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for n in (0, 1, 3, 40):
        out = k.run(num_ctas=n, status=status)
        torch.cuda.synchronize()
        check(out, ref, f"{name} ctas={n}")
        assert torch.equal(out, k.run(num_ctas=n)), "run-to-run results differ"
    assert int(status.item()) == 0


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (64, 0), (63, 64), (100, 5), (200, 129), (500, 1 << 20), (1 << 30, 2)])
@pytest.mark.parametrize("shape", [SHAPES[4], SHAPES[5], SHAPES[7]], ids=["ragged", "mixed_d256", "p48"])
def test_chunk_window_matches_reference(shape, window, sinks):
    name, qlens, ctx, Hq, Hkv, D, P = shape
    k = Chunk(name, qlens, ctx, Hq, Hkv, D, P, seed=72)
    ref = k.ref(window, sinks)
    for n in (0, 2):
        check(k.run(window, sinks, num_ctas=n), ref, f"{name} window={window} sinks={sinks} ctas={n}")


def test_chunk_agrees_with_the_other_attention_calls():
    k = Chunk("agree", [4, 4, 4], [900, 4, 2000], 24, 4, 256, 64)
    out = k.run().view(3, 4, 24, 256)
    q = k.q.view(3, 4, 24, 256)
    args = (k.c.bt, k.c.ctx, k.w.sm_scale, k.w.max_ctx)
    check(out, nk.paged_decode_attn(k.c.pool, q, *args).double(), "decode", roundings=2)
    check(out, nk.paged_prefill_attn(k.c.pool, q, *args).double(), "prefill", roundings=2)
    check(k.run(100, 4).view(3, 4, 24, 256), nk.paged_window_attn(k.c.pool, q, *args, 100, sinks=4).double(), "window",
          roundings=2)


@pytest.mark.parametrize("which,s", [("q", -12), ("q", 20), ("v", -30), ("v", 10), ("v", 60), ("k", 6), ("k", -40)])
def test_chunk_scaled_inputs(which, s):
    """The fp16 operands carry powers of two: inputs far from unit scale. (q x 2^20 is answered by k x 2^-20.)"""
    kw = {f"{which}_scale": 2.0 ** s}
    if (which, s) == ("q", 20):
        kw["k_scale"] = 2.0 ** -20
    k = Chunk(f"ck_{which}{s}", [96], [900], 24, 4, 256, 64, **kw)
    if which == "k" and s == 6:  # scores of some hundreds: the roundings move near-ties by their full weight
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        assert torch.isfinite(k.run(status=status)).all() and int(status.item()) == 0
        return
    check(k.run(), k.ref(), k.w.name, unit=2.0 ** s if which == "v" else 1.0)


def test_chunk_values_whose_scales_jump_between_blocks():
    """Each 64-token stretch of V 2^16 times as large or as small as the one before: the exponents move, the accumulator follows."""
    k = Chunk("jump", [70], [640], 8, 2, 128, 64)
    storage = k.c.pool.storage.view(k.w.num_pages, 2, -1)
    P, D = 64, 128
    vs = storage[..., 2 * P * D + P * 2 * 4:].view(torch.float32)
    for i, page in enumerate(k.c.bt[0, :10].tolist()):
        vs[page] *= 2.0 ** (16 * (i % 3) - 16)
    ref = k.ref()
    got = k.run().double()
    err = (got - ref).abs()
    # the weights reach over 32 powers of two: hold each element to the largest values it averages
    assert torch.all(err <= 2.0 ** -8 * ref.abs() + 4e-3 * 2.0 ** 16), float(err.max())
    assert float((got - ref).norm() / ref.norm()) <= 2.5e-3


def test_chunk_leaves_other_rows_and_flags_bad_sequences():
    k = Chunk("rows", [30, 20, 40, 10], [100, 200, 300, 50], 8, 2, 128, 16)
    ref = k.ref()
    q = torch.cat([k.q, k.q[:13]])  # rows behind the last sequence
    out = torch.full_like(q, 7.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    k.run(q=q, out=out, status=status)
    torch.cuda.synchronize()
    check(out[:100], ref, "rows")
    assert torch.all(out[100:] == 7.0) and int(status.item()) == 0
    ctx = k.c.ctx.clone()
    ctx[1], ctx[3] = 19, k.w.max_ctx + 1  # fewer tokens than the chunk has; more than the call allows
    out.fill_(7.0)
    k.run(q=q, out=out, ctx=ctx, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == nk.NK_DEVFLAG_BAD_CTX
    check(torch.cat([out[:30], out[50:90]]), torch.cat([ref[:30], ref[50:90]]), "valid sequences")
    assert torch.all(out[30:50] == 7.0) and torch.all(out[90:] == 7.0)
    cu = k.cu.clone()
    cu[2] = 20  # decreasing: sequence 1 has -10 rows, sequence 2 seventy (of its 300 tokens, not its own rows)
    cu[4] = 1 << 20
    out.fill_(7.0)
    status.zero_()
    k.run(q=q, out=out, cu=cu, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == nk.NK_DEVFLAG_BAD_CTX
    assert torch.all(out[90:] == 7.0)
    out.fill_(7.0)
    nk.paged_chunk_attn(k.c.pool, q, torch.zeros_like(k.cu), k.c.bt, k.c.ctx, k.w.sm_scale, k.w.max_ctx, out=out)
    torch.cuda.synchronize()
    assert torch.all(out == 7.0)


def test_chunk_bad_pages_and_non_finite_rows_are_flagged():
    k = Chunk("bad", [30, 30], [100, 200], 8, 2, 128, 16)
    ref = k.ref()
    bt = k.c.bt.clone()
    bt[0, 2], bt[0, 3] = -1, k.w.num_pages
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = k.run(bt=bt, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == nk.NK_DEVFLAG_BAD_PAGE and torch.isfinite(out).all()
    check(out[30:], ref[30:], "the other sequence")
    # a token whose value scale is infinite: no row before it is touched
    storage = k.c.pool.storage.view(k.w.num_pages, 2, -1)
    vs = storage[..., 2 * 16 * 128 + 16 * 2 * 4:].view(torch.float32).view(k.w.num_pages, 2, 16, 2)
    pos = 190
    vs[int(k.c.bt[1, pos // 16]), :, pos % 16] = float("inf")
    status.zero_()
    out = k.run(status=status)
    torch.cuda.synchronize()
    assert int(status.item()) & nk.NK_DEVFLAG_RANGE
    check(out[:50], ref[:50], "rows before the token")


def test_chunk_pages_outside_the_window_are_not_read():
    k = Chunk("freed", [70, 1], [2000, 1111], 24, 4, 256, 64)
    want = k.run(200, 70)
    bt = k.c.bt.clone()
    for b, (L, T) in enumerate(zip(k.w.ctx_lens, k.qlens)):
        bt[b, 2:(L - T - 200 + 1) // 64] = -1
        bt[b, -(-L // 64):] = 1 << 30
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = k.run(200, 70, bt=bt, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and torch.equal(out, want)


def test_chunk_many_sequences_and_graph_replay():
    rng = np.random.RandomState(3)
    ctx = rng.randint(1, 400, 1024).tolist()
    qlens = [int(rng.randint(0, min(L, 9) + 1)) for L in ctx]
    k = Chunk("many", qlens, ctx, 4, 2, 64, 16)
    check(k.run(), k.ref(), "1,024 sequences")
    want = k.run(50, 3)
    ws = torch.empty(nk.chunk_workspace_bytes(64), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        k.run(50, 3, workspace=ws, out=out)
    for _ in range(3):
        out.zero_()
        ws.fill_(0xFF)  # the workspace's contents on entry do not matter
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_chunk_wait_that_runs_out_is_reported():
    """The bounded waits (nk_test_inject_copy_stall): blocks from the third on are never handed to the tensor cores."""
    k = Chunk("stall", [20], [2000], 8, 2, 128, 64)
    want = k.run(num_ctas=2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    try:
        nk.test_inject_copy_stall(2, 2_000_000)
        k.run(num_ctas=2, status=status)
        torch.cuda.synchronize()
    finally:
        nk.test_inject_copy_stall(-1)
    assert int(status.item()) & nk.NK_DEVFLAG_TIMEOUT
    status.zero_()
    out = k.run(num_ctas=2, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and torch.equal(out, want)


@pytest.mark.parametrize("ctas", [1, 2, 5, 7, 0])
def test_chunk_tiles_dealt_out_whole_and_split(ctas):
    """More than two tiles a CTA: rounds of whole tiles, then split ones; tiles of very different lengths, sequences without
    tokens between them."""
    k = Chunk("rounds", [300, 0, 1, 1, 257, 0, 2, 128], [300, 7, 2500, 64, 1700, 90, 2, 1000], 8, 2, 64, 16, seed=77)
    for window, sinks in ((0, 0), (333, 5)):
        ref = k.ref(window, sinks)
        out = k.run(window, sinks, num_ctas=ctas)
        check(out, ref, f"ctas={ctas} window={window}")
        assert torch.equal(out, k.run(window, sinks, num_ctas=ctas))


def test_chunk_many_tiles_of_one_length():
    """The default split with rounds: 4 x 24 tiles a kv-head."""
    k = Chunk("even", [512] * 4, [1100, 700, 1024, 513], 20, 4, 128, 64, seed=78)
    check(k.run(), k.ref(), "rounds over the default CTAs")
