"""Operators of long contexts and of a verify round's end over the paged INT8 cache, as cases that can be timed and compared.

What a serving loop over a long cache needs beside the attention over all of it:
  bounds   per page and kv-head, the largest and smallest value of each key channel, in 8 bits, after the append of a step;
  select   the pages whose bounds promise the largest scores, chosen for each query token and kv-head;
  sparse   decode and verify attention (1 to 16 query tokens a sequence) over chosen pages only;
  weights  the attention weight that each page drew from a step's queries (or from the last 16 of a prompt), accumulated;
  evict    the pages with the least of it given back, block tables compacted;
  verify   drafted tokens accepted or replaced by the target's and the draft's probabilities and given random numbers.

``run`` computes each in elementary torch operations; with ``own`` set it calls this package. The cache is the package's
INT8 group-64 layout: pool[page][kv-head] holds Kc[P][D] int8 | Ks[P][D/64] fp32 | Vc[P][D] int8 | Vs[P][D/64] fp32. The
bounds are codes[page][kv-head][max, min][D] int8, then scales[page][kv-head] fp32.
"""
import math
import random

import torch

own = False

GROUP = 64


# ---------------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of eight conversations, each adds a token to its last page: latency
        dict(name="bounds_step8", op="bounds", B=8, Hkv=4, D=256, P=64, start_lo=500, start_hi=4000, new_lo=1, new_hi=1, mix=1),
        # the prompts of eight conversations, just appended
        dict(name="bounds_prompts", op="bounds", B=8, Hkv=4, D=256, P=64, start_lo=0, start_hi=0, new_lo=8000, new_hi=16384, mix=2),
        # one conversation at 262,144 tokens: 64 of its 4,096 pages
        dict(name="select_long1", op="select", B=1, T=1, Hq=24, Hkv=4, D=256, P=64, ctx_lo=262144, ctx_hi=262144, k=64, sinks=1, recent=2, mix=3),
        # a verify round of eight sequences
        dict(name="select_verify8", op="select", B=8, T=4, Hq=24, Hkv=4, D=256, P=64, ctx_lo=4096, ctx_hi=65536, k=64, sinks=1, recent=2, mix=4),
        # one conversation over 64 chosen pages: latency
        dict(name="sparse_long1", op="sparse", B=1, T=1, Hq=24, Hkv=4, D=256, P=64, ctx_lo=131072, ctx_hi=131072, k=64, mix=5),
        # a verify round of eight sequences, 4,096 keys for each of its tokens
        dict(name="sparse_verify8", op="sparse", B=8, T=4, Hq=24, Hkv=4, D=256, P=64, ctx_lo=4096, ctx_hi=65536, k=64, mix=6),
        # one decode step of one conversation: latency
        dict(name="weights_decode1", op="weights", B=1, T=1, Hq=24, Hkv=4, D=256, P=64, ctx_lo=32768, ctx_hi=32768, seen=True, mix=7),
        # the last 16 tokens of eight prompts look back over them, before a first eviction
        dict(name="weights_window8", op="weights", B=8, T=16, Hq=24, Hkv=4, D=256, P=64, ctx_lo=8192, ctx_hi=65536, seen=False, mix=8),
        # eight long conversations cut back to 16K tokens
        dict(name="evict_8", op="evict", B=8, Hkv=4, P=64, ctx_lo=32768, ctx_hi=131072, keep=256, sinks=1, recent=4, mix=9),
        # a large batch over small pages, most of them over their budget, two kv-heads
        dict(name="evict_batch512", op="evict", B=512, Hkv=2, P=16, ctx_lo=500, ctx_hi=20000, keep=125, sinks=1, recent=3, mix=10),
        # three drafts of one conversation, an odd vocabulary: latency
        dict(name="verify_1", op="verify", B=1, T=4, V=50001, ragged=False, draft=True, mix=11),
        # seven drafts of 64 conversations
        dict(name="verify_batch64", op="verify", B=64, T=8, V=131072, ragged=True, draft=True, mix=12),
    ]


HEADS = [(24, 4, 256), (8, 2, 256), (16, 2, 128), (32, 8, 128), (8, 8, 64), (10, 2, 64), (5, 5, 128), (14, 2, 256)]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["bounds", "select", "sparse", "weights", "evict", "verify"])
    mix = rng.randrange(1 << 20)
    Hq, Hkv, D = rng.choice(HEADS)
    P = rng.choice([16, 32, 48, 64, 128])
    if op == "bounds":
        B = _log(rng, 1, 64)
        lo, hi = _log(rng, 1, 4096), _log(rng, 1, 131072 // B)
        return dict(op=op, B=B, Hkv=Hkv, D=D, P=P, start_lo=0 if rng.random() < 0.3 else max(1, lo // 8), start_hi=lo, new_lo=max(1, hi // 4), new_hi=hi, mix=mix)
    if op == "verify":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, T=rng.choice([1, 2, 3, 4, 5, 8]), V=_log(rng, 64, 131072), ragged=rng.random() < 0.5, draft=rng.random() < 0.8, mix=mix)
    if op == "evict":
        B = _log(rng, 1, 512)
        hi = _log(rng, 64, min(131072, 4194304 // B))
        sinks, recent = rng.choice([0, 1, 2]), rng.choice([1, 2, 5])
        return dict(op=op, B=B, Hkv=Hkv, P=P, ctx_lo=max(1, hi // 16), ctx_hi=hi, keep=sinks + recent + _log(rng, 1, 512), sinks=sinks, recent=recent, mix=mix)
    T, B = rng.choice([1, 1, 1, 2, 3, 4, 5, 8, 16]), _log(rng, 1, 32)
    hi = _log(rng, 64, min(65536, 262144 // B))
    both = dict(op=op, B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, P=P, ctx_lo=max(T, hi // 8), ctx_hi=hi, mix=mix)
    if op == "weights":
        return both | dict(seen=rng.random() < 0.5)
    most = (1 << 27) // (B * T * Hkv * P * D)  # as many keys as the largest listed case reads
    k = _log(rng, 3, min(128, 8192 // P) if op == "select" else max(3, min(128, 8192 // P, most)))
    return both | dict(k=k) | (dict(sinks=rng.choice([0, 1]), recent=rng.choice([1, 2])) if op == "select" else {})


def _lens(case):
    """Two whole numbers a sequence: first positions and new tokens, or contexts and query tokens."""
    rng = random.Random(case["mix"])
    B = case["B"]
    if case["op"] == "bounds":
        start = [_log(rng, max(1, case["start_lo"]), case["start_hi"]) if case["start_hi"] else 0 for _ in range(B)]
        new = [case["new_hi"]] + [_log(rng, case["new_lo"], case["new_hi"]) for _ in range(B - 1)]
        if B > 4:  # a request that starts here, and one that brings nothing
            start[B // 2], new[B // 3] = 0, 0
        return start, new
    if case["op"] == "verify":
        T = case["T"]
        return [rng.randint(T, 65536) for _ in range(B)], [rng.randint(0, T - 1) if case["ragged"] else T - 1 for _ in range(B)]
    return [case["ctx_hi"]] + [_log(rng, case["ctx_lo"], case["ctx_hi"]) for _ in range(B - 1)], [case.get("T", 1)] * B


# -------------------------------------------------------------------------------------------------------------- prepare
def _chunk_bytes(P, D):
    return 2 * P * D + 2 * P * (D // GROUP) * 4


def _views(storage, pages, Hkv, P, D):
    """The codes [pages][Hkv][P][D] and scales [pages][Hkv][P][D/64] of K and V inside a pool's bytes."""
    chunk, sc = _chunk_bytes(P, D), P * (D // GROUP) * 4
    s = storage.view(pages, Hkv, chunk)
    part = lambda a, n, t, w: s[..., a:a + n].view(t).unflatten(-1, (P, w))  # noqa: E731
    return (part(0, P * D, torch.int8, D), part(P * D, sc, torch.float32, D // GROUP),
            part(P * D + sc, P * D, torch.int8, D), part(2 * P * D + sc, sc, torch.float32, D // GROUP))


def _bound_views(storage, pages, Hkv, D):
    """The codes [pages][Hkv][2][D] and scales [pages][Hkv] inside the bytes of a pool's bounds."""
    n = pages * Hkv * 2 * D
    return storage[:n].view(torch.int8).view(pages, Hkv, 2, D), storage[n:].view(torch.float32).view(pages, Hkv)


def _fill(storage, pages, Hkv, P, D, g):
    """Quantized rows of N(0, 1) in every slot; a few K channels are eight times as large, as real keys have them, and the
    keys of a page have a mean of their own, as neighbouring tokens' keys have."""
    kc, ks, vc, vs = _views(storage, pages, Hkv, P, D)
    wide = torch.ones(D, device="cuda")
    wide[torch.randperm(D, generator=g, device="cuda")[:4]] = 8.0
    step = max(1, (1 << 27) // (Hkv * P * D))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        for codes, scales, mul in ((kc, ks, wide), (vc, vs, None)):
            x = torch.randn((n, Hkv, P, D), generator=g, device="cuda")
            if mul is not None:
                x = (x + 0.5 * torch.randn((n, Hkv, 1, D), generator=g, device="cuda")) * mul
            x = x.to(torch.bfloat16).float().unflatten(-1, (D // GROUP, GROUP))
            s = x.abs().amax(-1) / 127
            codes[a:a + n] = (x / s[..., None]).round().clamp(-127, 127).to(torch.int8).flatten(-2)
            scales[a:a + n] = s


def _tables(held, g, spare=2):
    """Pages in all, and a block table whose sequences hold so many of them in random order (-1 behind)."""
    pages = sum(held) + spare
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(held), max(1, max(held))), -1, dtype=torch.int32, device="cuda")
    n = torch.tensor(held, device="cuda")[:, None]
    table[torch.arange(table.shape[1], device="cuda")[None] < n] = perm[:sum(held)]
    return pages, table


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, B = case["op"], case["B"]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    randn = lambda *n: torch.randn(n, generator=g, device="cuda")  # noqa: E731
    c127 = torch.full((), 127.0, device="cuda")  # a tensor: torch multiplies by the reciprocal of a number
    s = dict(case=case, status=i32([0]), c127=c127)
    first, second = _lens(case)
    if op == "verify":
        T, V = case["T"], case["V"]
        logits = randn(B, T, V) * 2.5
        p = torch.softmax(logits, -1)
        drafts = torch.zeros((B, max(0, T - 1)), dtype=torch.int32, device="cuda")
        q = None
        if T > 1:  # the draft model is near the target
            q = torch.softmax(logits[:, :T - 1] + 0.7 * randn(B, T - 1, V), -1)
            drafts = torch.multinomial(q.view(-1, V), 1, generator=g).view(B, T - 1).to(torch.int32)
        elif case["draft"]:
            q = torch.zeros((B, 0, V), device="cuda")
        return s | dict(p=p, q=q if case["draft"] else None, drafts=drafts, u=torch.rand((B, T), generator=g, device="cuda"),
                        count=i32(second) if case["ragged"] else None, n=i32(second), ctx=i32(first))
    Hkv, P = case["Hkv"], case["P"]
    if op == "bounds":
        D = case["D"]
        end = [a + n for a, n in zip(first, second)]
        pages, table = _tables([-(-e // P) for e in end], g)
        storage = torch.empty(pages * Hkv * _chunk_bytes(P, D), dtype=torch.uint8, device="cuda")
        _fill(storage, pages, Hkv, P, D, g)
        bounds = torch.zeros(pages * Hkv * (2 * D + 4), dtype=torch.uint8, device="cuda")
        cu = [0]
        for n in second:
            cu.append(cu[-1] + n)
        return s | dict(storage=storage, pages=pages, table=table, bounds=bounds, start=i32(first), end=i32(end), cu=i32(cu))
    held = [-(-n // P) for n in first]
    pages, table = _tables(held, g)
    s |= dict(pages=pages, table=table, ctx=i32(first), max_ctx=max(first))
    if op == "evict":
        # weight falls off as a power, as attention's does, the same in all of a page's heads but for a factor
        w = torch.rand((pages, 1), generator=g, device="cuda") ** 8 * torch.rand((pages, Hkv), generator=g, device="cuda")
        room = sum(max(0, h - case["keep"]) for h in held) + 3
        return s | dict(w=w, out=table.clone(), new_ctx=i32([0] * B), freed=i32([-7] * room), count=i32([0]))
    T, Hq, D = case["T"], case["Hq"], case["D"]
    s |= dict(q=randn(B, T, Hq, D).to(torch.bfloat16), scale=1 / math.sqrt(D))
    if op == "select":
        # the keys of a page spread about a mean of their own, as in _fill
        bounds = torch.empty(pages * Hkv * (2 * D + 4), dtype=torch.uint8, device="cuda")
        codes, scales = _bound_views(bounds, pages, Hkv, D)
        mid, width = 0.5 * randn(pages, Hkv, 1, D), 1.7 + 0.5 * randn(pages, Hkv, 2, D).abs()
        x = mid + width * torch.tensor([1.0, -1.0], device="cuda")[:, None]
        top = x.abs().amax((-1, -2)) / 127
        codes.copy_((x / top[..., None, None]).round().clamp(-127, 127))
        scales.copy_(top)
        return s | dict(bounds=bounds)
    s["storage"] = torch.empty(pages * Hkv * _chunk_bytes(P, D), dtype=torch.uint8, device="cuda")
    _fill(s["storage"], pages, Hkv, P, D, g)
    if op == "weights":
        prior = torch.rand((pages, Hkv), generator=g, device="cuda") if case["seen"] else None
        seen = i32([max(0, n - T) for n in first]) if case["seen"] else None
        return s | dict(prior=prior, seen=seen, out=torch.zeros((pages, Hkv), device="cuda"))
    # chosen pages: random ones of those that the token sees, its own last, in ascending order, -1 behind
    k, N = case["k"], table.shape[1]
    last = (i32(first)[:, None] - T + torch.arange(T, device="cuda")) // P  # [B][T]
    order = torch.rand((B, T, Hkv, N), generator=g, device="cuda")
    i = torch.arange(N, device="cuda")
    order = torch.where(i < last[..., None, None], order, torch.where(i == last[..., None, None], -1.0, 2.0))
    pick = order.argsort(-1)[..., :k]
    pick = torch.where(torch.gather(order, -1, pick) < 1.5, pick, 1 << 30).sort(-1).values
    chosen = torch.full((B, T, Hkv, k), -1, dtype=torch.int32, device="cuda")
    chosen[..., :pick.shape[-1]] = torch.where(pick < 1 << 30, pick, -1)
    return s | dict(chosen=chosen)


# ------------------------------------------------------------------------------------------------------------------ run
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    return {"bounds": _bounds, "select": _select, "sparse": _sparse, "weights": _weights, "evict": _evict, "verify": _verify}[op](s)


def _own(s, op):
    import quantized_paged_kv_cache_gb300 as nk

    c = s["case"]
    if op == "verify":
        next_start = torch.empty_like(s["ctx"])
        tokens, accepted = nk.verify_drafts(s["p"], s["q"], s["drafts"], s["u"], num_drafts=s["count"], ctx_lens=s["ctx"], next_start=next_start,
                                            status=s["status"])
        return tokens, accepted, next_start
    if op == "evict":
        nk.evict_pages(c["P"], s["w"], s["table"], s["ctx"], c["keep"], s["new_ctx"], s["freed"], s["count"], sink_pages=c["sinks"],
                       recent_pages=c["recent"], out=s["out"], status=s["status"])
        return s["out"], s["new_ctx"], s["freed"], s["count"]
    if op == "select":
        bounds = nk.PageBounds(s["bounds"], s["pages"], c["Hkv"], c["D"])
        return nk.page_select(bounds, s["q"], s["table"], s["ctx"], c["P"], s["max_ctx"], c["k"], sink_pages=c["sinks"], recent_pages=c["recent"],
                              status=s["status"])
    pool = nk.KVPool(s["storage"], s["pages"], c["P"], c["Hkv"], c["D"])
    if op == "bounds":
        bounds = nk.PageBounds(s["bounds"], s["pages"], c["Hkv"], c["D"])
        nk.page_bounds(pool, bounds, s["table"], s["start"], s["cu"], status=s["status"])
        return bounds.values()
    if op == "sparse":
        return nk.paged_sparse_attn(pool, s["q"], s["table"], s["ctx"], s["chosen"], s["scale"], s["max_ctx"], status=s["status"])
    return nk.page_weights(pool, s["q"], s["table"], s["ctx"], s["scale"], s["max_ctx"], s["out"], prior=s["prior"], seen=s["seen"], status=s["status"])


def _bounds(s):
    c = s["case"]
    P, D, Hkv = c["P"], c["D"], c["Hkv"]
    codes, scales = _bound_views(s["bounds"], s["pages"], Hkv, D)
    i = torch.arange(s["table"].shape[1], device="cuda")[None]
    touched = (i >= (s["start"] // P)[:, None]) & (i * P < s["end"][:, None]) & (s["end"] > s["start"])[:, None]
    page = torch.where(touched, s["table"], -1).flatten()
    live = torch.nonzero(page >= 0).flatten()
    page = page[live].long()
    filled = (s["end"][:, None] - i * P).flatten()[live]
    kc, ks, _, _ = _views(s["storage"], s["pages"], Hkv, P, D)
    x = (kc[page].float().unflatten(-1, (D // GROUP, GROUP)) * ks[page][..., None]).flatten(-2)
    empty = (torch.arange(P, device="cuda")[None] >= filled[:, None])[:, None, :, None]
    hi, lo = x.masked_fill(empty, -math.inf).amax(2), x.masked_fill(empty, math.inf).amin(2)
    both = torch.stack([hi, lo], 2)
    top = both.abs().amax((-1, -2)) / s["c127"]
    top = torch.where(top == 0, 1.0, top)
    codes[page] = (both / top[..., None, None]).round().clamp(-127, 127).to(torch.int8)
    scales[page] = top
    return codes.float() * scales[..., None, None]


def _select(s):
    c = s["case"]
    B, T, Hq, Hkv, D, P, k = (c[x] for x in ("B", "T", "Hq", "Hkv", "D", "P", "k"))
    codes, scales = _bound_views(s["bounds"], s["pages"], Hkv, D)
    N = s["table"].shape[1]
    q = s["q"].float().view(B, T, Hkv, Hq // Hkv, D)
    top = q.abs().amax((-1, -2), keepdim=True) / s["c127"]
    q = (q / torch.where(top == 0, 1.0, top)).round().clamp(-127, 127).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    page = s["table"].long().clamp(min=0)
    b8 = codes[page].float().permute(0, 2, 3, 4, 1)  # [B][Hkv][2][D][N]
    whole = q.clamp(min=0) @ b8[:, :, 0] + q.clamp(max=0) @ b8[:, :, 1]  # whole numbers below 2^24: exact in 32 bits
    score = whole.view(B, Hkv, T, Hq // Hkv, N).amax(3).double() * scales[page].double().permute(0, 2, 1)[:, :, None]
    seen = ((s["ctx"].long()[:, None] - T + torch.arange(T, device="cuda")) // P + 1)[:, None, :, None]
    i = torch.arange(N, device="cuda")
    score = torch.where((i < c["sinks"]) | (i >= seen - c["recent"]), math.inf, score)
    score = torch.where(i < seen, score, -math.inf)
    best, pick = score.sort(dim=-1, descending=True, stable=True)
    pick = torch.where(best > -math.inf, pick, 1 << 30)[..., :k].sort(-1).values
    out = torch.full((B, T, Hkv, k), -1, dtype=torch.int32, device="cuda")
    out[..., :pick.shape[-1]] = torch.where(pick < 1 << 30, pick, -1).permute(0, 2, 1, 3)
    return out


def _sparse(s):
    c = s["case"]
    B, T, Hq, Hkv, D, P, k = (c[x] for x in ("B", "T", "Hq", "Hkv", "D", "P", "k"))
    chosen = s["chosen"].long()  # [B][T][Hkv][k]
    there = chosen >= 0
    page = torch.gather(s["table"].long(), 1, chosen.clamp(min=0).view(B, -1)).view(chosen.shape)
    page = torch.where(there, page, 0)
    head = torch.arange(Hkv, device="cuda")[:, None]
    rows = lambda codes, scales: (codes[page, head].float().unflatten(-1, (D // GROUP, GROUP)) * scales[page, head][..., None]).flatten(-2).flatten(3, 4)  # noqa: E731
    kc, ks, vc, vs = _views(s["storage"], s["pages"], Hkv, P, D)
    key = (chosen[..., None] * P + torch.arange(P, device="cuda")).flatten(-2)
    pos = (s["ctx"].long()[:, None] - T + torch.arange(T, device="cuda"))[:, :, None, None]
    seen = there.repeat_interleave(P, -1) & (key <= pos)
    score = (s["q"].float().view(B, T, Hkv, Hq // Hkv, D) @ rows(kc, ks).transpose(-1, -2)).mul_(s["scale"])
    score.masked_fill_(~seen[..., None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(top == -math.inf, 0, top)).exp_()
    total = score.sum(-1, keepdim=True)
    out = (score @ rows(vc, vs)) / torch.where(total == 0, 1, total)
    return out.reshape(B, T, Hq, D).to(torch.bfloat16)


def _weights(s):
    c = s["case"]
    B, T, Hq, Hkv, D, P = (c[x] for x in ("B", "T", "Hq", "Hkv", "D", "P"))
    N = s["table"].shape[1]
    page = s["table"].long().clamp(min=0)
    kc, ks, _, _ = _views(s["storage"], s["pages"], Hkv, P, D)
    k = (kc[page].float().unflatten(-1, (D // GROUP, GROUP)) * ks[page][..., None]).flatten(-2)  # [B][N][Hkv][P][D]
    q = s["q"].float().view(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    score = (q @ k.permute(0, 2, 4, 1, 3).reshape(B, Hkv, D, N * P)).mul_(s["scale"]).view(B, Hkv, T, Hq // Hkv, N * P)
    pos = s["ctx"].long()[:, None] - T + torch.arange(T, device="cuda")
    hidden = torch.arange(N * P, device="cuda") > pos[..., None]
    score.masked_fill_(hidden[:, None, :, None], -math.inf)
    score.sub_(score.amax(-1, keepdim=True)).exp_()
    score.div_(score.sum(-1, keepdim=True))
    mass = score.view(B, Hkv, -1, N, P).sum((2, 4)).transpose(1, 2)  # [B][N][Hkv]
    live = torch.arange(N, device="cuda")[None] * P < s["ctx"][:, None]
    if s["prior"] is not None:
        old = torch.arange(N, device="cuda")[None] * P < s["seen"][:, None]
        mass = mass + torch.where(old[..., None], s["prior"][page], 0)
    s["out"][page[live]] = mass[live]
    return s["out"]


def _evict(s):
    c = s["case"]
    P, keep = c["P"], c["keep"]
    N = s["table"].shape[1]
    held = ((s["ctx"].long() + P - 1) // P)[:, None]
    i = torch.arange(N, device="cuda")[None]
    w = s["w"].double()[s["table"].long().clamp(min=0)].sum(-1)
    w = torch.where((i < c["sinks"]) | (i >= held - c["recent"]), math.inf, w)
    w = torch.where(i < held, w, -math.inf)
    order = w.sort(dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, i.expand_as(order))
    kept = (rank < keep) & (i < held)
    gone = (i < held) & ~kept
    at = kept.cumsum(1) - 1
    out = torch.where(i < held, -1, s["table"])
    b = torch.arange(out.shape[0], device="cuda")[:, None].expand_as(out)
    out[b[kept], at[kept]] = s["table"][kept]
    free = s["table"][gone]
    s["freed"][:free.numel()] = free
    return out, (s["ctx"].long() - P * gone.sum(1)).int(), s["freed"], gone.sum().int()[None]


def _verify(s):
    p, q, drafts, n = s["p"], s["q"], s["drafts"].long(), s["n"].long()
    B, T, V = p.shape
    b, t = torch.arange(B, device="cuda"), torch.arange(T, device="cuda")[None]
    px = torch.gather(p[:, :T - 1], 2, drafts[..., None])[..., 0]
    qx = torch.gather(q, 2, drafts[..., None])[..., 0] if q is not None else torch.ones_like(px)
    good = (s["u"][:, :T - 1].double() * qx.double() < px.double()) & (t[:, :T - 1] < n[:, None])
    a = good.long().cumprod(1).sum(1)
    row, cut = p[b, a], a < n
    if T > 1:
        at = a.clamp(max=T - 2)
        minus = q[b, at] if q is not None else (torch.arange(V, device="cuda")[None] == drafts[b, at][:, None]).float() * row
        rest = (row - torch.where(cut[:, None], minus, 0)).clamp(min=0)
        rest = torch.where(rest.double().sum(1, keepdim=True) > 0, rest, row)
    else:
        rest = row
    cdf = rest.double().cumsum(1)
    token = (cdf <= s["u"][:, T - 1:].double() * cdf[:, -1:]).sum(1)
    before = torch.cat([drafts, drafts.new_zeros((B, 1))], 1)
    tokens = torch.where(t < a[:, None], before, torch.where(t == a[:, None], token[:, None], -1))
    return tokens.int(), a.int(), (s["ctx"].long() - n + a).int()


# ---------------------------------------------------------------------------------------------------------------- exact
def exact(case, seed):
    op = case["op"]
    if op in ("select", "evict", "verify"):
        return None  # whole numbers
    s = prepare(case, seed)
    Hkv, D, P, B = case["Hkv"], case["D"], case["P"], case["B"]
    sc = P * D // GROUP * 4
    pool = s["storage"].view(s["pages"], Hkv, -1)

    def dequantized(page, h, a):  # of one head, [pages * P][D], in 64 bits
        raw = pool[page, h]
        code = raw[:, a:a + P * D].contiguous().view(torch.int8).reshape(-1, D // GROUP, GROUP).double()
        return (code * raw[:, a + P * D:a + P * D + sc].contiguous().view(torch.float32).reshape(-1, D // GROUP, 1).double()).reshape(-1, D)

    if op == "bounds":
        start, new = _lens(case)
        out = torch.zeros((s["pages"], Hkv, 2, D), dtype=torch.float64, device="cuda")
        for b in range(B):
            if not new[b]:
                continue
            first, end = start[b] // P, start[b] + new[b]
            page = s["table"][b, first:-(-end // P)].long()
            for h in range(Hkv):
                x = dequantized(page, h, 0).float().double()  # a value, a scale and a quotient are each rounded once to 32 bits
                n = end - first * P
                last = x[(page.numel() - 1) * P:n]
                full = x[:(page.numel() - 1) * P].view(-1, P, D)
                both = torch.stack([torch.cat([full.amax(1), last.amax(0)[None]]), torch.cat([full.amin(1), last.amin(0)[None]])], 1)
                top = (both.abs().amax((1, 2)) / 127).float().double()
                top = torch.where(top == 0, torch.ones_like(top), top)[:, None, None]
                out[page, h] = torch.round((both / top).float().double()).clamp(-127, 127) * top
        return out
    ctx, _ = _lens(case)
    T, Hq = case["T"], case["Hq"]
    G = Hq // Hkv
    q = s["q"].double()
    if op == "weights":
        out = torch.zeros((s["pages"], Hkv), dtype=torch.float64, device="cuda")
        for b, L in enumerate(ctx):
            page = s["table"][b, :-(-L // P)].long()
            hidden = torch.arange(L, device="cuda")[None] > torch.arange(L - T, L, device="cuda")[:, None]
            for h in range(Hkv):
                kt = dequantized(page, h, 0)[:L].T
                mass = torch.zeros(page.numel() * P, dtype=torch.float64, device="cuda")
                for i in range(h * G, h * G + G):
                    mass[:L] += torch.softmax((q[b, :, i] @ kt / math.sqrt(D)).masked_fill(hidden, -math.inf), -1).sum(0)
                out[page, h] = mass.view(-1, P).sum(1)
                if s["prior"] is not None:
                    old = -(-int(s["seen"][b]) // P)
                    out[page[:old], h] += s["prior"][page[:old], h].double()
        return out
    if B * T * Hkv > 1024:
        return None
    out = torch.zeros_like(q)
    chosen, table = s["chosen"].cpu(), s["table"].cpu()
    for b, L in enumerate(ctx):
        for t in range(T):
            for h in range(Hkv):
                mine = chosen[b, t, h]
                mine = mine[mine >= 0].long()
                page = table[b, mine].long().cuda()
                key = (mine[:, None] * P + torch.arange(P)).flatten().cuda()
                e = q[b, t, h * G:h * G + G] @ dequantized(page, h, 0).T / math.sqrt(D)
                e = e.masked_fill(key[None] > L - T + t, -math.inf)
                out[b, t, h * G:h * G + G] = torch.softmax(e, -1) @ dequantized(page, h, P * D + sc)
    return out


# ----------------------------------------------------------------------------------------------------------------- work
def work(case):
    op, B = case["op"], case["B"]
    first, second = _lens(case)
    if op == "verify":  # the drafts' probabilities, and one row of each side, of the target's alone where nothing was drafted
        rows = sum(2 if n and case["draft"] else 1 for n in second)
        return {"bytes": rows * case["V"] * 4 + sum(second) * 16 + B * (4 + 4 * case["T"] + 12), "flops": sum(second) * 2 + 2 * rows * case["V"]}
    P, Hkv = case["P"], case["Hkv"]
    if op == "evict":
        held = [-(-n // P) for n in first]
        return {"bytes": sum(held) * (4 * Hkv + 8) + 8 * B, "flops": sum(held) * Hkv}
    D = case["D"]
    half = D + D // GROUP * 4  # a key (or a value) of one head, with its scales
    if op == "bounds":
        ends = [(a // P * P, a + n) for a, n in zip(first, second) if n]
        keys, pages = sum(e - a for a, e in ends), sum(-(-(e - a) // P) for a, e in ends)
        return {"bytes": Hkv * (keys * half + pages * (2 * D + 4)) + 8 * B + 4 * pages, "flops": 3 * keys * Hkv * D}
    T, Hq = case["T"], case["Hq"]
    rows = B * T * Hq * D * 2
    if op == "select":
        pages = sum(-(-n // P) for n in first if -(-n // P) > case["k"])  # shorter ones have nothing to choose
        return {"bytes": rows + pages * (Hkv * (2 * D + 4) + 4) + B * T * Hkv * case["k"] * 4, "flops": 2 * pages * T * Hq * D}
    if op == "weights":
        pages = sum(-(-n // P) for n in first)
        return {"bytes": rows + sum(first) * Hkv * half + pages * (4 + Hkv * (8 if case["seen"] else 4)), "flops": 2 * sum(first) * T * Hq * D}
    keys = sum(min(-(-(n - T + t + 1) // P), case["k"]) * P - (-(n - T + t + 1) % P) for n in first for t in range(T))
    read = sum(min(T * min(-(-n // P), case["k"]) * P, n) for n in first)  # pages that several tokens chose are read once, at best
    return {"bytes": 2 * rows + read * Hkv * 2 * half + B * T * Hkv * case["k"] * 4, "flops": 4 * keys * Hq * D}
