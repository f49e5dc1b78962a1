"""Plain forms of the operators over long caches and of draft verification, one
page, key and token at a time in 64 bits, for the tests of their kernels.
Nothing here is shared with the library; the pool's and the bounds' bytes are
read by the documented layouts. Where the definitions round to fp32 (a value of
the cache, a scale, a quotient, a difference of probabilities), so do these."""
from __future__ import annotations

import numpy as np
import torch

import _ref


def f32(x):
    return np.asarray(x, dtype=np.float64).astype(np.float32).astype(np.float64)


def rows(codes, scales):
    """fp32 values of [..., D] codes and [..., D/64] scales, as fp64 (non-finite scales as zeros)."""
    s = np.where(np.isfinite(scales), scales, 0).astype(np.float64)
    return f32(codes.astype(np.float64).reshape(*codes.shape[:-1], -1, 64) * s[..., None]).reshape(codes.shape)


def keys(storage, num_pages, Hkv, P, D):
    """(codes int8 [pages][Hkv][P][D], scales fp32 [pages][Hkv][P][D/64]) of the pool's keys."""
    raw = storage.cpu().numpy().reshape(num_pages, Hkv, -1)
    n, sc = P * D, P * (D // 64) * 4
    return (raw[..., :n].copy().view(np.int8).reshape(num_pages, Hkv, P, D),
            raw[..., n:n + sc].copy().view(np.float32).reshape(num_pages, Hkv, P, D // 64))


def round_half_even(x):
    return np.clip(np.rint(x), -127, 127)


def bounds(kc, ks, page, filled):
    """(codes int8 [Hkv][2][D], scales fp32 [Hkv]) of one page."""
    v = rows(kc[page, :, :filled], ks[page, :, :filled])
    both = np.stack([v.max(1), v.min(1)], 1)
    s = f32(np.abs(both).max((1, 2)) / 127)
    s = np.where(s == 0, 1.0, s)
    return round_half_even(f32(both / s[:, None, None])).astype(np.int8), s.astype(np.float32)


def select(codes, scales, q, table, ctx, P, k, sinks, recent):
    """int32 [B][T][Hkv][k]; codes [pages][Hkv][2][D], q fp64 [B][T][Hq][D]. Scores are whole numbers (Python's) times
    the exact value of the fp32 scale."""
    B, T, Hq, D = q.shape
    Hkv = codes.shape[1]
    G = Hq // Hkv
    out = np.full((B, T, Hkv, k), -1, np.int32)
    for b in range(B):
        for t in range(T):
            seen = (ctx[b] - T + t) // P + 1
            for h in range(Hkv):
                x = q[b, t, h * G:(h + 1) * G]
                if not np.isfinite(x).all():
                    x = np.zeros_like(x)
                s = float(f32(np.abs(x).max() / 127)) or 1.0
                q8 = round_half_even(f32(x / s)).astype(np.int64)
                pages = list(range(seen))
                if seen > k:
                    always = set(range(sinks)) | set(range(seen - recent, seen))
                    score = []
                    for i in pages:
                        page = table[b, i]
                        ok = 0 <= page < codes.shape[0] and i not in always and np.isfinite(scales[page, h])
                        if not ok:
                            score.append(-1e308)
                            continue
                        c = codes[page, h].astype(np.int64)
                        whole = (np.maximum(q8, 0) @ c[0] + np.minimum(q8, 0) @ c[1]).max()
                        score.append(float(int(whole)) * float(scales[page, h]))  # (23 + 24 bits: exact)
                    rest = sorted((i for i in pages if i not in always), key=lambda i: (-score[i], i))
                    pages = sorted(always | set(rest[:k - len(always)]))
                out[b, t, h, :len(pages)] = pages
    return out


def sparse(storage, num_pages, Hkv, P, D, table, ctx, lists, q, sm_scale):
    """fp64 [B][T][Hq][D]: attention over the listed pages' visible keys; zeros where there are none."""
    K, V = (x.cpu().numpy() for x in _ref.dequantized(storage, num_pages, Hkv, P, D))
    q = q.double().cpu().numpy()
    B, T, Hq, _ = q.shape
    G = Hq // Hkv
    out = np.zeros_like(q)
    for b in range(B):
        for t in range(T):
            pos = ctx[b] - T + t
            for h in range(Hkv):
                ks, vs = [], []
                for i in lists[b, t, h]:
                    if 0 <= i <= pos // P:
                        n = min(P, pos + 1 - i * P)
                        ks.append(K[table[b, i], h, :n])
                        vs.append(V[table[b, i], h, :n])
                if not ks:
                    continue
                k, v = np.concatenate(ks), np.concatenate(vs)
                s = q[b, t, h * G:(h + 1) * G] @ k.T * sm_scale
                e = np.exp(s - s.max(-1, keepdims=True))
                out[b, t, h * G:(h + 1) * G] = e @ v / e.sum(-1, keepdims=True)
    return out


def weights(storage, num_pages, Hkv, P, D, table, ctx, q, sm_scale):
    """{(page, h): weight} in fp64."""
    K = _ref.dequantized(storage, num_pages, Hkv, P, D)[0].cpu().numpy()
    q = q.double().cpu().numpy()
    B, T, Hq, _ = q.shape
    G = Hq // Hkv
    out = {}
    for b in range(B):
        n = -(-ctx[b] // P)
        for h in range(Hkv):
            k = K[table[b, :n], h].reshape(n * P, D)[:ctx[b]]
            mass = np.zeros(n * P)
            for t in range(T):
                s = q[b, t, h * G:(h + 1) * G] @ k[:ctx[b] - T + t + 1].T * sm_scale
                e = np.exp(s - s.max(-1, keepdims=True))
                mass[:e.shape[1]] += (e / e.sum(-1, keepdims=True)).sum(0)
            for i, m in enumerate(mass.reshape(n, P).sum(1)):
                out[int(table[b, i]), h] = m
    return out


def evict(w, table, ctx, P, keep, sinks, recent):
    """(table, lengths, freed pages); sums as exact fractions of the fp32 weights."""
    from fractions import Fraction

    table, lens, freed = table.copy(), [], []
    for b, L in enumerate(ctx):
        n = -(-L // P)
        if n <= keep:
            lens.append(L)
            continue
        row = table[b, :n].copy()
        total = [sum((Fraction(float(x)) for x in w[p]), Fraction(0)) for p in row]
        always = set(range(sinks)) | set(range(n - recent, n))
        rest = sorted((i for i in range(n) if i not in always), key=lambda i: (-total[i], i))
        kept = sorted(always | set(rest[:keep - len(always)]))
        freed += [int(row[i]) for i in range(n) if i not in set(kept)]
        table[b, :n] = -1
        table[b, :len(kept)] = row[kept]
        lens.append(L - P * (n - len(kept)))
    return table, lens, freed


def verify(p, q, drafts, u, num=None):
    """(tokens [B][T], accepted [B]); p fp32 [B][T][V], q [B][T-1][V] or None; sums as whole multiples of 2^-149."""
    B, T, V = p.shape
    tokens, accepted = np.full((B, T), -1, np.int64), []
    one = 2.0 ** 149

    def whole(x):  # fp32 values as whole numbers, exactly
        return [int(v * 2.0 ** 100) * 2 ** 49 if v >= 2.0 ** -60 else int(v * one) for v in x.astype(np.float64)]

    for b in range(B):
        n = T - 1 if num is None else int(num[b])
        a = 0
        while a < n:
            x = int(drafts[b, a])
            if not 0 <= x < V:
                break
            qx = 1.0 if q is None else float(q[b, a, x])
            if not float(u[b, a]) * qx < float(p[b, a, x]):
                break
            tokens[b, a] = x
            a += 1
        row = p[b, a]
        r = row
        if a < n:
            if q is None:
                r = row.copy()
                r[int(drafts[b, a])] = 0
            else:
                r = (row - q[b, a]).astype(np.float32)
            r = np.maximum(r, 0)
            if not (r > 0).any():
                r = row
        r = np.clip(np.nan_to_num(r, nan=0.0), 0, 1)
        w = whole(r)
        total = sum(w)
        ut = float(u[b, T - 1])
        ut = min(max(ut, 0.0), 1 - 2.0 ** -24) if ut == ut else 0.0
        num_u, run = int(ut * 2.0 ** 149) if ut < 2.0 ** -60 else int(ut * 2.0 ** 100) * 2 ** 49, 0
        for i, x in enumerate(w):
            run += x
            if run * 2 ** 149 > num_u * total:
                tokens[b, a] = i
                break
        accepted.append(a)
    return tokens, np.array(accepted)
