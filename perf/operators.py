"""The operators around one serving step over the paged INT8 cache, as cases that can be timed and compared.

A step of a serving loop with continuous batching needs, beside the cache's append and decode:
  tables  the block tables and slot maps of the step, built on the GPU from the requests' lengths and a list of free pages;
  mrope   the rotation of its query and key rows by positions with several axes (time, height, width);
  window  decode and verify attention (1 to 16 query tokens a sequence) over a sliding window and a few first tokens (sinks);
  chunk   attention of ragged chunks of new tokens (one token to thousands a sequence), over everything before them or a window.

``run`` computes each in elementary torch operations, in 32 bits; with ``own`` set it calls this package. The cache is
the package's INT8 group-64 layout: pool[page][kv-head] holds Kc[P][D] int8 | Ks[P][D/64] fp32 | Vc[P][D] int8 | Vs[P][D/64] fp32.
"""
import math
import random

import torch

own = False

GROUP = 64


# ---------------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of eight long conversations: latency
        dict(name="tables_step8", op="tables", B=8, P=64, start_lo=4096, start_hi=65536, new_lo=1, new_hi=1, mix=1),
        # a large ragged batch whose requests bring prompts and chunks of up to 1,024 tokens
        dict(name="tables_ragged1024", op="tables", B=1024, P=64, start_lo=1, start_hi=16384, new_lo=1, new_hi=1024, mix=2),
        # the query and key rows of one decode step of eight sequences: latency
        dict(name="mrope_step8", op="mrope", rows=8, Hq=24, Hkv=4, D=256, rot=256, s1=48, s2=48, interleaved=False, far=65536),
        # eight chunks of 1,024 tokens
        dict(name="mrope_chunk8192", op="mrope", rows=8192, Hq=24, Hkv=4, D=256, rot=256, s1=48, s2=48, interleaved=False, far=131072),
        # half of each head rotated, axes dealt out in turn, an odd number of rows, far positions
        dict(name="mrope_partial", op="mrope", rows=4099, Hq=16, Hkv=2, D=128, rot=64, s1=10, s2=10, interleaved=True, far=262144),
        # one conversation at 32K with a 4,096-token window and four sinks: latency
        dict(name="window_decode1", op="window", B=1, T=1, Hq=24, Hkv=4, D=256, P=64, ctx_lo=32768, ctx_hi=32768, W=4096, S=4, mix=3),
        # a verify round of eight sequences, a wide window
        dict(name="window_verify8", op="window", B=8, T=4, Hq=24, Hkv=4, D=256, P=64, ctx_lo=4096, ctx_hi=65536, W=8192, S=64, mix=4),
        # many short windows over small pages, odd window and sink lengths
        dict(name="window_batch64", op="window", B=64, T=1, Hq=16, Hkv=2, D=128, P=16, ctx_lo=100, ctx_hi=20000, W=1000, S=5, mix=5),
        # the rest of one short prompt: few rows, latency
        dict(name="chunk_small", op="chunk", B=1, single=0, q_lo=77, q_hi=77, Hq=16, Hkv=2, D=128, P=16, ctx_lo=1500, ctx_hi=1500, W=0, S=0, mix=6),
        # continuous batching: twelve sequences decode one token while four bring chunks
        dict(name="chunk_mixed16", op="chunk", B=16, single=12, q_lo=64, q_hi=1024, Hq=24, Hkv=4, D=256, P=64, ctx_lo=1024, ctx_hi=32768, W=0, S=0, mix=7),
        # chunks of 1,024 tokens in a model with a 4,096-token window and four sinks
        dict(name="chunk_window4", op="chunk", B=4, single=0, q_lo=1024, q_hi=1024, Hq=24, Hkv=4, D=256, P=64, ctx_lo=8192, ctx_hi=32768, W=4096, S=4, mix=8),
        # chunked prefill of eight sequences, 1,024 tokens each, at up to 32K
        dict(name="chunk_8x1024", op="chunk", B=8, single=0, q_lo=1024, q_hi=1024, Hq=24, Hkv=4, D=256, P=64, ctx_lo=8192, ctx_hi=32768, W=0, S=0, mix=9),
    ]


HEADS = [(24, 4, 256), (8, 2, 256), (16, 2, 128), (32, 8, 128), (8, 8, 64), (10, 2, 64), (5, 5, 128), (14, 2, 256)]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["tables", "mrope", "window", "chunk"])
    mix = rng.randrange(1 << 20)
    Hq, Hkv, D = rng.choice(HEADS)
    if op == "tables":
        B = _log(rng, 1, 1024)
        return dict(op=op, B=B, P=rng.choice([16, 32, 48, 64, 128, 256]), start_lo=1, start_hi=_log(rng, 1, min(131072, 16777216 // B)),
                    new_lo=1, new_hi=_log(rng, 1, 1024), mix=mix)
    if op == "mrope":
        rot = rng.choice([D, D // 2])
        s1 = rng.randint(0, rot // 6)
        return dict(op=op, rows=_log(rng, 1, 8192), Hq=Hq, Hkv=Hkv, D=D, rot=rot, s1=s1, s2=rng.randint(0, rot // 6),
                    interleaved=rng.random() < 0.5, far=_log(rng, 16, 262144))
    P = rng.choice([16, 32, 48, 64, 128])
    if op == "window":
        T, B = rng.choice([1, 1, 1, 2, 3, 4, 5, 8, 16]), _log(rng, 1, 64)
        hi = _log(rng, 64, min(65536, 524288 // B))
        W = _log(rng, 1, min(hi, 16384))
        return dict(op=op, B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, P=P, ctx_lo=max(T, hi // 8), ctx_hi=hi, W=W, S=rng.choice([0, 1, 4, 5, 64, 130]), mix=mix)
    B = _log(rng, 1, 16)
    hi = _log(rng, 64, 32768)
    q_hi = min(hi, _log(rng, 1, min(1024, 8192 // B)))
    windowed = rng.random() < 0.4
    return dict(op=op, B=B, single=rng.randint(0, B - 1) if rng.random() < 0.5 else 0, q_lo=max(1, q_hi // 8), q_hi=q_hi, Hq=Hq, Hkv=Hkv, D=D,
                P=P, ctx_lo=max(q_hi, hi // 8), ctx_hi=hi, W=_log(rng, 1, 8192) if windowed else 0, S=rng.choice([0, 1, 4, 64]) if windowed else 0, mix=mix)


def _lens(case):
    """(first positions or contexts, new or query tokens) of the case's sequences."""
    rng = random.Random(case["mix"])
    B = case["B"]
    if case["op"] == "tables":
        start = [_log(rng, case["start_lo"], case["start_hi"]) for _ in range(B)]
        new = [_log(rng, case["new_lo"], case["new_hi"]) for _ in range(B)]
        if B > 4:  # a request that starts here, and one that brings nothing
            start[B // 2], new[B // 3] = 0, 0
        return start, new
    ctx = [case["ctx_hi"]] + [_log(rng, case["ctx_lo"], case["ctx_hi"]) for _ in range(B - 1)]
    if case["op"] == "window":
        return ctx, [case["T"]] * B
    q = [case["q_hi"]] + [_log(rng, case["q_lo"], case["q_hi"]) for _ in range(B - 1)]
    for b in range(B - case["single"], B):
        q[b] = 1
    return ctx, [min(t, n) for t, n in zip(q, ctx)]


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


def _fill(storage, pages, Hkv, P, D, g):
    """Quantized rows of N(0, 1) in every slot; a few K channels are eight times as large, as real keys have them."""
    kc, ks, vc, vs = _views(storage, pages, Hkv, P, D)
    wide = torch.ones(D, device="cuda")
    wide[torch.randperm(D, generator=g, device="cuda")[:4]] = 8.0
    step = max(1, (1 << 27) // (Hkv * P * D))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        for codes, scales, mul in ((kc, ks, wide), (vc, vs, None)):
            x = torch.randn((n, Hkv, P, D), generator=g, device="cuda")
            x = (x if mul is None else x * mul).to(torch.bfloat16).float().unflatten(-1, (D // GROUP, GROUP))
            s = x.abs().amax(-1) / 127
            codes[a:a + n] = (x / s[..., None]).round().clamp(-127, 127).to(torch.int8).flatten(-2)
            scales[a:a + n] = s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if case["op"] == "tables":
        P, B = case["P"], case["B"]
        start, new = _lens(case)
        old = [-(-s // P) for s in start]
        need = [-(-(s + n) // P) - o for s, n, o in zip(start, new, old)]
        pages = sum(old) + sum(need) + 8
        perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        width = max(o + n for o, n in zip(old, need)) + 1
        table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        held = torch.arange(width, device="cuda")[None] < i32(old)[:, None]
        table[held] = perm[:sum(old)]
        rows = sum(new) + 3  # a step's buffers are sized for the largest step: rows behind the last sequence stay
        return dict(case=case, P=P, pages=pages, start=i32(start), new=i32(new), free=perm[sum(old):].clone(), table=table, rows=rows,
                    cu=i32([0] * (B + 1)), ctx=i32([0] * B), slots=torch.full((rows,), -7, dtype=torch.int64, device="cuda"),
                    positions=torch.full((rows,), -7, dtype=torch.int32, device="cuda"), used=i32([0]), status=status)
    if case["op"] == "mrope":
        n, Hq, Hkv, D, rot = (case[k] for k in ("rows", "Hq", "Hkv", "D", "rot"))
        # rows of one fused projection: queries, keys and values of a token side by side
        qkv = torch.randn((n, Hq + 2 * Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
        t = torch.randint(0, case["far"], (1,), generator=g, device="cuda") + torch.arange(n, device="cuda")
        hw = torch.randint(0, 64, (2, n), generator=g, device="cuda")
        pos = torch.stack([t, t + hw[0], t + hw[1]]).to(torch.int32)
        inv = 1e6 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)
        sections = (rot // 2 - case["s1"] - case["s2"], case["s1"], case["s2"])
        return dict(case=case, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], pos=pos, inv=inv, inv_cuda=inv.cuda(), sections=sections,
                    axis=_axes(sections, case["interleaved"]).cuda())
    Hq, Hkv, D, P, B = (case[k] for k in ("Hq", "Hkv", "D", "P", "B"))
    ctx, q = _lens(case)
    held = [-(-n // P) for n in ctx]
    pages = sum(held) + 2
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, max(held)), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(max(held), device="cuda")[None] < i32(held)[:, None]] = perm[:sum(held)]
    storage = torch.empty(pages * Hkv * _chunk_bytes(P, D), dtype=torch.uint8, device="cuda")
    _fill(storage, pages, Hkv, P, D, g)
    cu = [0]
    for t in q:
        cu.append(cu[-1] + t)
    x = torch.randn((cu[-1], Hq, D), generator=g, device="cuda").to(torch.bfloat16)
    W, S = (case["W"], case["S"]) if case["W"] else (1 << 30, 0)
    Tm = max(q)
    return dict(case=case, storage=storage, pages=pages, table=table, ctx=i32(ctx), qlen=i32(q), cu=i32(cu), max_ctx=max(ctx), Tm=Tm, W=W, S=S, scale=1 / math.sqrt(D), status=status,
                q=x.view(B, case["T"], Hq, D) if case["op"] == "window" else x)


def _axes(sections, interleaved):
    """The axis (0 time, 1 height, 2 width) of each frequency: one run of frequencies after another, or the axes in turn."""
    n = sum(sections)
    if not interleaved:
        return torch.repeat_interleave(torch.arange(3), torch.tensor(sections))
    i = torch.arange(n)
    return torch.where(i < 3 * torch.tensor(sections)[i % 3], i % 3, torch.zeros_like(i))


# ------------------------------------------------------------------------------------------------------------------ run
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    return {"tables": _tables, "mrope": _mrope, "window": _window, "chunk": _chunk}[op](s)


def _own(s, op):
    import quantized_paged_kv_cache_gb300 as nk

    c = s["case"]
    if op == "tables":
        nk.step_tables(s["P"], s["pages"], s["start"], s["new"], s["free"], s["table"], s["cu"], s["ctx"], s["slots"], positions=s["positions"],
                       used=s["used"], status=s["status"])
        return s["table"], s["cu"], s["ctx"], s["slots"], s["positions"], s["used"]
    if op == "mrope":
        return nk.mrope(s["q"], s["k"], s["pos"], s["inv"], s["sections"], interleaved=c["interleaved"])
    pool = nk.KVPool(s["storage"], s["pages"], c["P"], c["Hkv"], c["D"])
    if op == "window":
        return nk.paged_window_attn(pool, s["q"], s["table"], s["ctx"], s["scale"], s["max_ctx"], s["W"], sinks=s["S"], status=s["status"])
    return nk.paged_chunk_attn(pool, s["q"], s["cu"], s["table"], s["ctx"], s["scale"], s["max_ctx"], window=c["W"], sinks=c["S"], status=s["status"])


def _tables(s):
    P, start, new, table, free = s["P"], s["start"].long(), s["new"].long(), s["table"], s["free"]
    B, width = table.shape
    cu = torch.zeros(B + 1, dtype=torch.int64, device="cuda")
    cu[1:] = new.cumsum(0)
    first, last = (start + P - 1) // P, (start + new + P - 1) // P
    need = last - first
    off = need.cumsum(0) - need
    i = torch.arange(width, device="cuda")[None]
    fresh = (i >= first[:, None]) & (i < last[:, None])
    pick = (off[:, None] + i - first[:, None]).clamp(0, free.numel() - 1)
    table.copy_(torch.where(fresh, free[pick], table))
    j = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(cu[1:], j, right=True).clamp(max=B - 1)
    live = j < cu[B]
    pos = start[b] + j - cu[b]
    slot = table[b, (pos // P).clamp(max=width - 1)].long() * P + pos % P
    s["slots"].copy_(torch.where(live, slot, s["slots"]))
    s["positions"].copy_(torch.where(live, pos.int(), s["positions"]))
    return table, cu.int(), (start + new).int(), s["slots"], s["positions"], need.sum().int()[None]


def _mrope(s):
    rot = s["case"]["rot"]
    angle = s["pos"].double()[s["axis"]].T * s["inv_cuda"]  # 64 bits: 32 lose a far position's angle
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turn(x):
        x = x.float()
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], -1).to(torch.bfloat16)

    return turn(s["q"]), turn(s["k"])


def _attend(s, q, of=slice(None)):
    """Attention of q [B][Tm][Hq][D] (the own tokens of each of the sequences `of` first) over the cached keys that they see; fp32, as q."""
    c = s["case"]
    Hq, Hkv, D, P = (c[k] for k in ("Hq", "Hkv", "D", "P"))
    B, Tm, W, S = q.shape[0], q.shape[1], s["W"], s["S"]
    ctx, qlen = s["ctx"][of].long(), s["qlen"][of].long()
    lo = (ctx - qlen - W + 1).clamp(min=0)  # the first key inside any of the sequence's windows
    n = torch.arange(min(s["max_ctx"], S + W + Tm - 1), device="cuda")[None]
    lead = lo.clamp(max=S)[:, None]  # sinks before it
    key = torch.where(n < lead, n, n - lead + lo[:, None])
    there = key < ctx[:, None]
    key = torch.where(there, key, 0)
    page, slot = torch.gather(s["table"][of].long(), 1, key // P), key % P
    kc, ks, vc, vs = _views(s["storage"], s["pages"], Hkv, P, D)
    rows = lambda codes, scales: (codes[page, :, slot].float().unflatten(-1, (D // GROUP, GROUP)) * scales[page, :, slot][..., None]).flatten(-2)  # noqa: E731
    k, v = rows(kc, ks).transpose(1, 2), rows(vc, vs).transpose(1, 2)  # [B][Hkv][keys][D]
    x = q.float().view(B, Tm, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    score = (x @ k.transpose(-1, -2)).mul_(s["scale"]).view(B, Hkv, Hq // Hkv, Tm, -1)
    pos = (ctx - qlen)[:, None] + torch.arange(Tm, device="cuda")[None]
    key = key[:, None]
    seen = there[:, None] & (key <= pos[..., None]) & ((key > pos[..., None] - W) | (key < S))
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(top == -math.inf, 0, top)).exp_()
    total = score.sum(-1, keepdim=True)
    out = score.view(B, Hkv, -1, score.shape[-1]) @ v
    return (out.view(B, Hkv, Hq // Hkv, Tm, D) / total).permute(0, 3, 1, 2, 4).reshape(B, Tm, Hq, D)


def _window(s):
    return _attend(s, s["q"]).to(torch.bfloat16)


def _chunk(s):
    # the chunks are padded to the longest; the sequences with a single token, the last ones, are a batch of their own
    q, cu, one = s["q"], s["cu"].long(), s["case"]["single"]
    B, rows = cu.numel() - 1 - one, q.shape[0] - one
    t = torch.arange(s["Tm"], device="cuda")[None]
    at = (cu[:B, None] + t).clamp(max=rows - 1)
    j = torch.arange(rows, device="cuda")
    b = torch.searchsorted(cu[1:B + 1], j, right=True)
    out = _attend(s, q[at], slice(0, B))[b, j - cu[b]]
    if one:
        out = torch.cat([out, _attend(s, q[rows:, None], slice(B, None))[:, 0]])
    return out.to(torch.bfloat16)


# ---------------------------------------------------------------------------------------------------------------- exact
def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "mrope":
        half = case["rot"] // 2
        axis = _axes(s["sections"], case["interleaved"]).tolist()
        z = []
        for x in (s["q"], s["k"]):
            y = x.double()
            for i in range(half):
                w = s["pos"][axis[i]].double() * 1e6 ** (-2.0 * i / case["rot"])
                turned = torch.view_as_complex(torch.stack([x[..., i], x[..., i + half]], -1).double()) * torch.polar(torch.ones_like(w), w)[:, None]
                y[..., i], y[..., i + half] = turned.real, turned.imag
            z.append(y)
        return tuple(z)
    ctx, qlen = _lens(case)
    Hq, Hkv, D, P = (case[k] for k in ("Hq", "Hkv", "D", "P"))
    pool = s["storage"].view(s["pages"], Hkv, -1)
    scales = P * D // GROUP * 4
    q = s["q"].reshape(-1, Hq, D).double()
    out = torch.empty_like(q)
    at = 0
    for b, (L, T) in enumerate(zip(ctx, qlen)):
        pages = s["table"][b, :-(-L // P)].long()
        lo = max(0, L - T - s["W"] + 1)
        keys = torch.cat([torch.arange(min(s["S"], lo)), torch.arange(lo, L)]).cuda()
        pos = torch.arange(L - T, L, device="cuda")[:, None]
        hidden = (keys > pos) | ((keys <= pos - s["W"]) & (keys >= s["S"]))
        for h in range(Hkv):
            raw = pool[pages, h]
            kv = []
            for a in (0, P * D + scales):
                code = raw[:, a:a + P * D].contiguous().view(torch.int8).reshape(-1, D // GROUP, GROUP)[keys].double()
                scale = raw[:, a + P * D:a + P * D + scales].contiguous().view(torch.float32).reshape(-1, D // GROUP, 1)[keys].double()
                kv.append((code * scale).reshape(-1, D))
            for i in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                e = (q[at:at + T, i] @ kv[0].T / math.sqrt(D)).masked_fill_(hidden, -math.inf)
                out[at:at + T, i] = torch.softmax(e, -1) @ kv[1]
        at += T
    return out.view(s["q"].shape)


# ----------------------------------------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "mrope":
        n, heads = case["rows"], case["Hq"] + case["Hkv"]
        return {"bytes": n * (heads * case["D"] * 4 + 12), "flops": n * heads * case["rot"] * 3}
    ctx, q = _lens(case)
    B, P = case["B"], case["P"]
    if case["op"] == "tables":
        need = sum(-(-(s + n) // P) + -s // P for s, n in zip(ctx, q))
        return {"bytes": 4 * (2 * B + 2 * B + 2) + 8 * need + 12 * sum(q) + 4 * B, "flops": 2 * sum(q) + 4 * B}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    W, S = (case["W"], case["S"]) if case["W"] else (1 << 30, 0)
    read = pairs = 0
    for L, T in zip(ctx, q):
        lo = max(0, L - T - W + 1)
        read += L - lo + min(S, lo)
        # keys of the token at position p: its window, and the sinks before that
        if W >= L:
            pairs += T * (2 * L - T + 1) // 2
        else:
            pairs += sum(min(p + 1, W) + min(S, max(0, p + 1 - W)) for p in range(L - T, L))
    return {"bytes": read * Hkv * (2 * D + 2 * (D // GROUP) * 4) + 4 * sum(q) * Hq * D, "flops": 4 * D * Hq * pairs}
