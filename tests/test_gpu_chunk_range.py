"""nk_paged_chunk_attn on caches whose keys and channel groups differ widely in size, and with all-zero ones among them:
against the plain 64-bit form over the pool's own bytes.

The roundings (half a step each): the output to bf16, 2^-8 of the value; code * fp16(scale) in fp16, 2^-11 each of the value,
or, for values far below the largest of the 16 keys they share an exponent with, 2^-20 of that largest; a weight in fp16,
2^-11 of it, or 2^-32 of the reference weight (that of a key at most 2^8 below the row's largest; fp16's half step of 2^-25
is 2^-32 of it, because it is held as 2^7). Scores enter as in test_gpu_chunk.py; where only values are looked at, q is zero and the scores are
exact."""
import math

import pytest
import torch

import quantized_paged_kv_cache_gb300 as nk

import _ref
from test_gpu_chunk import check

pytestmark = pytest.mark.gpu


class Cache:
    """One sequence whose rows [L][Hkv][D] went through the append; the last T tokens are the chunk."""

    def __init__(self, k, v, q, P=64, window=0, sinks=0):
        L, self.Hkv, self.D = k.shape
        self.P, self.L, self.T, self.q, self.window, self.sinks = P, L, q.shape[0], q.bfloat16(), window, sinks
        self.pages = -(-L // P) + 1
        self.pool = nk.KVPool.empty(self.pages, P, self.Hkv, self.D)
        self.pool.storage.fill_(0xFF)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.bt = torch.arange(self.pages - 1, -1, -1, dtype=torch.int32, device="cuda")[:-1].view(1, -1).contiguous()
        self.ctx, self.cu = i32([L]), i32([0, self.T])
        nk.kv_append(self.pool, self.bt, i32([0]), i32([0, L]), k.bfloat16(), v.bfloat16())
        self.scale = 1 / math.sqrt(self.D)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def parts(self):
        """The pool's scales of K and V, [pages][Hkv][P][D/64], writable."""
        raw = self.pool.storage.view(self.pages, self.Hkv, -1)
        n, sc = self.P * self.D, self.P * (self.D // 64) * 4
        return [raw[..., a:a + sc].view(torch.float32).unflatten(-1, (self.P, self.D // 64)) for a in (n, 2 * n + sc)]

    def run(self, **kw):
        return nk.paged_chunk_attn(self.pool, self.q, self.cu, kw.pop("bt", self.bt), self.ctx, self.scale, self.L,
                                   window=self.window, sinks=self.sinks, status=self.status, **kw)

    def ref(self):
        return _ref.attention(self.pool.storage, self.pages, self.Hkv, self.P, self.D, self.bt, [self.L], [self.T], self.q,
                              self.scale, self.window, self.sinks)


def rows(seed, L, T, Hq, Hkv, D):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return r(L, Hkv, D), r(L, Hkv, D), r(T, Hq, D)


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("s", [-3, -6, -12, -30])
@pytest.mark.parametrize("D,P", [(64, 16), (128, 64), (256, 48), (256, 64)])
def test_zero_tokens_and_zero_channel_groups(which, s, D, P):
    """The append gives an all-zero group the scale 1: it must not set the exponent of the small rows beside it, whether the
    zero row is visible or still to come."""
    k, v, q = rows(5, 300, 40, 8, 2, D)
    unit = 1.0
    if which == "k":
        k, q = k * 2.0 ** s, q * 2.0 ** -s
    else:
        v, unit = v * 2.0 ** s, 2.0 ** s
    x = k if which == "k" else v
    x[7::16] = 0       # a token of every 16
    x[290:293] = 0     # hidden from most of the chunk's rows
    x[100:140, 1] = 0  # two whole groups of 16 keys of one kv-head
    if D > 64:
        x[3::5, :, 64:128] = 0  # a channel group of a fifth of the tokens
        x[:, 0, :64] = 0        # a channel group that is dead throughout
    c = Cache(k, v, q, P)
    check(c.run(), c.ref(), f"{which} 2^{s}", unit=unit)
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("which", [0, 1])
def test_groups_whose_scale_is_not_finite_count_as_zeros(which, value):
    k, v, q = rows(6, 200, 100, 8, 2, 128)
    c = Cache(k, v, q, 16)
    pos = 150
    x = c.parts()[which][int(c.bt[0, pos // 16]), :, pos % 16]
    x[:, 1] = 0.0
    want = c.ref()
    x[:, 1] = value
    out = c.run()
    torch.cuda.synchronize()
    assert int(c.status.item()) == nk.NK_DEVFLAG_RANGE
    check(out, want, f"{value}")


def test_groups_with_a_negative_scale():
    k, v, q = rows(7, 200, 50, 8, 2, 128)
    c = Cache(k, v, q, 16)
    for x in c.parts():
        x[:, :, 3:9] *= -1.0
        x[:, :, 12] *= -4.0
    # One key in 16 has K and V rows of four times N(0, 1): its score is off by four times the 5e-4 that the 4e-3 of `check`
    # stand on, and moves O by that times a |v - O| four times as large, so the bound is 4 * 4 times the one for unit rows.
    check(c.run(), c.ref(), "negative scales", unit=16.0)
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("r", [8, 12, 16, 20, 24, 40])
@pytest.mark.parametrize("G", [1, 6])
def test_a_row_does_not_see_the_size_of_hidden_keys(r, G):
    """Later tokens, and tokens before the window, whose values are 2^r times as large (in 16 keys of their own)."""
    k, v, q = rows(8, 128, 64, 4 * G, 4, 256)
    v[112:] *= 2.0 ** r
    c = Cache(k, v, q)
    ref = c.ref()
    check(c.run()[:48], ref[:48], "later tokens")
    check(c.run()[48:], ref[48:], "the tokens themselves", unit=2.0 ** r)
    v[112:] *= 2.0 ** -r
    v[:80] *= 2.0 ** r
    c = Cache(k, v, q, window=20)  # rows from position 99 on see none of the first 80 tokens
    check(c.run()[36:], c.ref()[36:], "tokens before the window")
    c = Cache(k, v, q, window=20, sinks=3)  # sinks among the loud ones: what the row sees is loud
    check(c.run(), c.ref(), "loud sinks", unit=2.0 ** r)
    assert int(c.status.item()) == 0


def test_values_that_fall_by_more_than_the_fp32_range():
    """V from 2^100 down to 2^-100: what the early blocks left must not overflow while the later ones are added."""
    k, v, q = rows(9, 64 * 5, 8, 8, 2, 128)
    for i, e in enumerate((100, -100, 0, -100, -20)):
        v[64 * i:64 * i + 64] *= 2.0 ** e
    c = Cache(k, v, q)
    check(c.run(num_ctas=1), c.ref(), "falling values", unit=2.0 ** 100)
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("r", [4, 8, 11, 12, 13, 14])
@pytest.mark.parametrize("loud", ["group", "key"])
def test_neighbours_of_different_size(loud, r):
    """Channel groups, or keys, of one 16 whose values differ by 2^r. The first token sees itself alone, the second itself
    and the first: nothing averages the roundings out."""
    L, Hkv, D = 64, 2, 256
    k, v, _ = rows(10 + r, L, L, 2, Hkv, D)
    if loud == "group":
        v[:, :, 64:128] *= 2.0 ** r
        quiet = [g for g in range(4) if g != 1]
    else:
        v[15::16] *= 2.0 ** r
        quiet = range(4)
    c = Cache(k, v, torch.zeros(L, 2, D, device="cuda"))
    K, V = _ref.dequantized(c.pool.storage, c.pages, Hkv, c.P, D)
    ref, out = c.ref(), c.run().double()
    V = V[int(c.bt[0, 0])]                                                 # [Hkv][64][D]
    largest = V.abs().amax(-1).view(Hkv, 4, 16).amax(-1)                   # of each 16 keys
    mean = lambda x: x.cumsum(1) / torch.arange(1, L + 1, device="cuda")[:, None]  # noqa: E731  (equal weights)
    near = mean(largest.repeat_interleave(16, 1)[..., None].expand(Hkv, L, 1)).transpose(0, 1)
    bound = 2.0 ** -8 * ref.abs() + 3 * 2.0 ** -11 * mean(V.abs()).transpose(0, 1) + 2.0 ** -20 * near
    err = (out - ref).abs()
    # (the weights' own step, for the largest value of all: 64 keys of 2^-32)
    bound = bound + 64 * 2.0 ** -32 * float(largest.max())
    assert torch.all(err <= bound), f"{loud} 2^{r}: {float((err - bound).max()):.3e} past the bound"
    first = out[0].view(Hkv, 4, 64)[:, list(quiet)], ref[0].view(Hkv, 4, 64)[:, list(quiet)]
    rel = float((first[0] - first[1]).norm() / first[1].norm())
    # bf16 1.65e-3, three fp16 roundings; 2^-25 of the operand's unit twice, uniform: 2^-20 2^r (4 sigma) / sqrt(12) at most
    assert rel <= math.hypot(2.5e-3, 2.0 ** (r - 18) / math.sqrt(12)), f"{loud} 2^{r}: relative norm {rel:.3e}"


@pytest.mark.parametrize("D", [128, 256])
def test_scores_beside_a_loud_channel_group_of_k(D):
    """K with a channel group 2^8 times as large as the others, which q leaves out. The operand of a quiet channel is off by
    two half steps of 2^-25 where the largest is 2^-3 at least: of rows of N(0, 1), with that largest at four times 2^8, by
    2^-24 2^3 4 2^8 / sqrt(12) = 2^-12.8 in the mean square, less than the 2^-11 sqrt(2/3) that `check` allows for already."""
    k, v, q = rows(12, 300, 60, 8, 2, D)
    k[:, :, 64:128] *= 2.0 ** 8
    q[:, :, 64:128] = 0
    c = Cache(k, v, q)
    check(c.run(), c.ref(), "loud group of K")
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("octaves", [20, 25, 26, 28])
@pytest.mark.parametrize("where", [0, 40000])
def test_many_keys_far_below_one_dominant_key(octaves, where):
    """131,072 keys whose weights lie 2^-octaves below one key's, which has no value: their sum is the result. The head's
    row 127 * 2^-k and the zero rows are exact in the cache, so the scores are, too: sm_scale * 256 * 127 * 2^-k * q."""
    L, D = 131072, 256
    k = torch.zeros(L, 1, D, device="cuda")
    k[where] = 127 * 2.0 ** -10
    v = torch.rand(L, 1, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)) * 0.25 + 0.75
    v[where] = 0
    qv = octaves * math.log(2) / (256 * 127 * 2.0 ** -10 / 16)
    q = torch.full((1, 2, D), qv, device="cuda")
    c = Cache(k, v, q)
    ref, out = c.ref(), c.run(num_ctas=1).double()  # (one CTA: its own sums meet the dominant key)
    # each weight is off by at most 2^-32 of the dominant one (half a step of fp16, which holds that one as 2^7), all of them
    # the same way here. The rest: bf16, V's and the scale's fp16 roundings.
    p = 2.0 ** -(octaves * float(q.bfloat16()[0, 0, 0]) / qv)
    tol = 2.0 ** -8 + 2.0 ** -32 / p + 3 * 2.0 ** -11 + 1e-3
    rel = float(((out - ref).abs() / ref).max())
    assert rel <= tol, f"relative error {rel:.3e}, bound {tol:.3e}"
