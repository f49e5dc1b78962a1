"""Verification of drafted tokens (nk_verify_drafts) against exact whole-number
arithmetic: tokens and counts must be equal."""
import numpy as np
import pytest
import torch

import quantized_paged_kv_cache_gb300 as nk

import _long_ref as ref

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def case(B, T, V, seed, near=0.7, temper=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((B, T, V), generator=g, device="cuda") * temper
    p = torch.softmax(x, -1)
    q = torch.softmax(x[:, :T - 1] + near * torch.randn((B, T - 1, V), generator=g, device="cuda"), -1)
    d = torch.multinomial(q.reshape(-1, V), 1, generator=g).view(B, T - 1).to(torch.int32) if T > 1 else i32(np.zeros((B, 0)))
    return p, q, d, torch.rand((B, T), generator=g, device="cuda")


def check(p, q, d, u, num=None, flags=0, **kw):
    B, T, V = p.shape
    status = i32([0])
    ctx, nxt = i32(np.arange(B) + 100), i32([-5] * B)
    tokens, acc = nk.verify_drafts(p, q, d, u, num_drafts=None if num is None else i32(num), ctx_lens=ctx, next_start=nxt, status=status, **kw)
    want, want_acc = ref.verify(p.cpu().numpy(), None if q is None else q.cpu().numpy(), d.cpu().numpy(), u.cpu().numpy(), num)
    assert acc.tolist() == want_acc.tolist()
    assert np.array_equal(tokens.cpu().numpy(), want)
    n = np.full(B, T - 1) if num is None else np.asarray(num)
    assert nxt.tolist() == (np.arange(B) + 100 - n + want_acc).tolist()
    assert int(status.item()) == flags
    return tokens, acc


@pytest.mark.parametrize("B,T,V", [(1, 1, 1), (1, 4, 50001), (5, 2, 7), (3, 16, 1000), (9, 3, 64), (2, 8, 4097), (70, 5, 333), (1, 3, 262147)])
@pytest.mark.parametrize("certain", [False, True])
def test_verify(B, T, V, certain):
    p, q, d, u = case(B, T, V, 7 * V + T)
    if certain:
        q = None
    check(p, q, d, u)
    check(p, q, d, u, num=[(3 * b) % T for b in range(B)])


@pytest.mark.parametrize("V", [40004, 65536, 131072])
@pytest.mark.parametrize("draft", ["certain", "aligned", "odd_rows"])
def test_aligned_rows(V, draft):
    """Rows that are read in pieces of four; with one side's rows off their 16 bytes; a refused draft of a large weight."""
    p, q, d, u = case(3, 3, V, V)
    p[:, 0] *= 0.6
    p[:, 0].scatter_(1, d[:, :1].long(), 0.4)
    u[:, 0] = torch.tensor([0.999999, 0.1, 0.999999], device="cuda")
    if draft == "certain":
        q = None
    elif draft == "odd_rows":
        q = torch.nn.functional.pad(q, (0, 1), value=float("nan"))[..., :V]
    for last in (1 / 7, 0.7, 1 - 2.0 ** -24):
        u[:, 2] = last
        check(p, q, d, u)


def test_acceptance_is_exact():
    """Products next to the target's probability: the rounded product equal to it, the exact one a half step aside; tiny ones."""
    rng = np.random.default_rng(31)
    n, V = 4000, 4
    u = (rng.random((n, 2)) * (1 - 2.0 ** -24)).astype(np.float32)
    qx = (rng.random(n) * 2.0 ** rng.choice([0, -1, -20, -70, -126], n)).astype(np.float32)
    u[:, 0] *= rng.choice(np.float32([1, 2.0 ** -10, 2.0 ** -60]), n)
    px = (u[:, 0].astype(np.float64) * qx).astype(np.float32)  # the rounded product
    px = np.where(np.arange(n) % 5 == 0, np.nextafter(px, np.float32(1)), px)
    px = np.where(np.arange(n) % 7 == 0, np.nextafter(px, np.float32(0)), px)
    p, q = np.full((n, 2, V), 0.25, np.float32), np.full((n, 1, V), 0.25, np.float32)
    p[:, 0, 2], q[:, 0, 2] = px, qx
    p, q, u = (torch.from_numpy(x).cuda() for x in (p, q, u))
    _, acc = nk.verify_drafts(p, q, i32(np.full((n, 1), 2)), u)
    want = u[:, 0].double() * q[:, 0, 2].double() < p[:, 0, 2].double()
    assert torch.equal(acc.bool(), want) and 0.2 < want.double().mean() < 0.8


def test_all_accepted_and_none():
    p, q, d, u = case(6, 4, 500, 3)
    same = p[:, :3].contiguous()
    _, acc = check(p, same, d, u * 0.99)  # the draft is the target: every ratio is 1
    assert acc.tolist() == [3] * 6
    u[:, :3] = 0.9999
    few = p.clone()
    few[:, :3].scatter_(2, d[..., None].long(), 1e-8)
    _, acc = check(few, q, d, u)
    assert acc.tolist() == [0] * 6


def test_uniforms_at_the_ends():
    """0 takes the first token that has a weight, the largest number below 1 the last one."""
    p, q, d, u = case(4, 1, 100, 5)
    p[:, :, :9] = 0
    p[:, :, 95:] = 0
    p[2:, :, 9:50] = 0
    u[0::2], u[1::2] = 0.0, 1 - 2.0 ** -24
    t, _ = check(p, None, d, u)
    assert t[:, 0].tolist() == [9, 94, 50, 94]
    u[:] = torch.tensor([[float("nan")], [2.0], [-1.0], [1.0]], device="cuda")  # outside: the nearest inside
    t, _ = check(p, None, d, u)
    assert t[:, 0].tolist() == [9, 94, 50, 94]


def test_uniforms_outside_decide_as_the_nearest_inside():
    p, _, d, u = case(4, 2, 100, 6)
    p[:, 0].scatter_(1, d.long(), torch.tensor([[0.5], [0.0], [0.0], [0.5]], device="cuda"))
    same = p[:, :1].clone().scatter_(2, d[..., None].long(), 0.5)
    u[:, 0] = torch.tensor([1.0, -1.0, float("nan"), float("nan")], device="cuda")
    _, acc = nk.verify_drafts(p, same, d, u)
    assert acc.tolist() == [1, 0, 0, 1]  # (1 - 2^-24) 0.5 < 0.5; 0 < 0 is not


def test_sums_that_32_bits_lose():
    """A hundred thousand equal weights below a large one: token i from u = (0.5 + i w) / R, between two of them."""
    V = 100001
    p = torch.full((8, 1, V), 2.0 ** -18, device="cuda")
    p[:, :, 0] = 0.5
    u = torch.tensor([(0.5 + (i + 0.5) * 2.0 ** -18) / (0.5 + (V - 1) * 2.0 ** -18) for i in (0, 1, 777, 5000, 33333, 50000, 77777, V - 2)],
                     dtype=torch.float64).float().cuda()[:, None]
    check(p, None, i32(np.zeros((8, 0))), u)


def test_nothing_left_after_the_draft_draws_from_the_target():
    p, q, d, u = case(4, 2, 300, 9)
    big = torch.clamp(p[:, :1] * 1.5, max=1.0).contiguous()  # above p everywhere
    u[:, 0] = 0.99
    _, acc = check(p, big, d, u)
    assert acc.tolist() == [0] * 4


def test_rows_without_a_distribution():
    p, q, d, u = case(5, 3, 200, 11)
    u[:, :2] = 0.0  # all accepted where p > 0
    p[1, 2] = 0.0
    p[2, 2, 5], p[2, 2, 6] = float("nan"), -1.0  # count as zero
    p[3, 2] = 0.5  # sums to 100
    status = i32([0])
    tokens, acc = nk.verify_drafts(p, q, d, u, status=status)
    assert int(status.item()) == nk.NK_DEVFLAG_RANGE and acc.tolist() == [2] * 5
    assert tokens[1, 2] == -1 and tokens[3, 2] == -1
    ok = [0, 2, 4]
    want, _ = ref.verify(p.cpu().numpy()[ok], q.cpu().numpy()[ok], d.cpu().numpy()[ok], u.cpu().numpy()[ok])
    assert np.array_equal(tokens.cpu().numpy()[ok], want)


def test_bad_drafts_and_counts():
    p, q, d, u = case(4, 4, 100, 13)
    d[0, 1], d[1, 0] = -1, 100
    check(p, q, d, u * 0, flags=nk.NK_DEVFLAG_BAD_TOKEN)
    p, q, d, u = case(4, 4, 100, 14)
    status, acc = i32([0]), i32([0] * 4)
    tokens, _ = nk.verify_drafts(p, q, d, u * 0, num_drafts=i32([-2, 9, 3, 1]), accepted=acc, status=status)
    assert int(status.item()) == nk.NK_DEVFLAG_BAD_POS
    want, n = ref.verify(p.cpu().numpy(), q.cpu().numpy(), d.cpu().numpy(), u.cpu().numpy() * 0, [0, 3, 3, 1])
    assert acc.tolist() == n.tolist() and np.array_equal(tokens.cpu().numpy(), want)


def test_padded_rows_streams_and_graphs():
    B, T, V = 3, 3, 1001
    p, q, d, u = case(B, T, V, 15)
    pad = torch.full((B, T, V + 23), float("nan"), device="cuda")
    pad[..., :V] = p
    qpad = torch.full((B, T - 1, V + 7), float("nan"), device="cuda")
    qpad[..., :V] = q
    want, acc = check(p, q, d, u)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got, a2 = nk.verify_drafts(pad[..., :V], qpad[..., :V], d, u, stream=st)
    st.synchronize()
    assert torch.equal(got, want) and torch.equal(a2, acc)
    tokens, accepted, g = torch.empty_like(want), torch.empty_like(acc), torch.cuda.CUDAGraph()
    ctx = i32([50] * B)
    with torch.cuda.graph(g):
        nk.verify_drafts(p, q, d, u, tokens=tokens, accepted=accepted, ctx_lens=ctx, next_start=ctx)  # in place
    g.replay()
    assert torch.equal(tokens, want) and ctx.tolist() == (48 + acc).tolist()
    # other numbers in the same graph
    u.copy_(torch.rand(u.shape, device="cuda"))
    ctx.fill_(50)
    g.replay()
    want, acc = ref.verify(p.cpu().numpy(), q.cpu().numpy(), d.cpu().numpy(), u.cpu().numpy())
    assert np.array_equal(tokens.cpu().numpy(), want) and accepted.tolist() == acc.tolist()
    with pytest.raises(ValueError):
        nk.verify_drafts(pad.transpose(0, 1)[..., :V], qpad[..., :V], d, u)
