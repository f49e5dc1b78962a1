"""Plain 64-bit forms of the step operators, for the tests of their kernels:
attention of ragged chunks over the paged INT8 cache with a window and sinks,
rotary positions with several axes, and the step's tables. Nothing here is
shared with the library; the pool's bytes are read by the documented layout."""
from __future__ import annotations

import math

import numpy as np
import torch


def dequantized(storage, num_pages, Hkv, P, D):
    """(K, V) of every slot, fp64 [num_pages][Hkv][P][D]."""
    raw = storage.reshape(num_pages, Hkv, -1)
    sc = P * (D // 64) * 4
    out = []
    for a in (0, P * D + sc):
        codes = raw[..., a:a + P * D].contiguous().view(torch.int8).reshape(num_pages, Hkv, P, D // 64, 64).double()
        scale = raw[..., a + P * D:a + P * D + sc].contiguous().view(torch.float32).reshape(num_pages, Hkv, P, D // 64, 1)
        out.append((codes * scale.double()).reshape(num_pages, Hkv, P, D))
    return out


def attention(storage, num_pages, Hkv, P, D, table, ctx, qlens, q, sm_scale, window=0, sinks=0):
    """fp64 [total][Hq][D]: token t of sequence b, at position p = ctx - qlen + t,
    sees key n <= p when window is 0, n > p - window or n < sinks."""
    K, V = dequantized(storage, num_pages, Hkv, P, D)
    Hq = q.shape[-2]
    q = q.reshape(-1, Hq, D).double()
    out = torch.zeros_like(q)
    at = 0
    for b, (L, T) in enumerate(zip(ctx, qlens)):
        if T == 0:
            continue
        n = torch.arange(L, device=q.device)
        pos = torch.arange(L - T, L, device=q.device)[:, None]
        seen = n <= pos
        if window > 0:
            seen &= (n > pos - window) | (n < sinks)
        need = seen.any(0)
        keys = n[need]  # keys nobody sees may lie in pages that were given back
        page = table[b].to(q.device).long()[keys // P]
        for h in range(Hkv):
            k, v = K[page, h, keys % P], V[page, h, keys % P]
            for i in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                s = (q[at:at + T, i] @ k.T) * sm_scale
                s.masked_fill_(~seen[:, need], -math.inf)
                out[at:at + T, i] = torch.softmax(s, -1) @ v
        at += T
    return out


def mrope(x, positions, inv_freq, sections, interleaved):
    """fp64 rotation of x [rows][heads][D]; also |a| + |b| of each element's pair (0 where it is copied)."""
    half = len(inv_freq)
    y = x.double().clone()
    size = torch.zeros_like(y)
    axes, A = [], len(sections)
    if interleaved:
        axes = [i % A if i < A * sections[i % A] else 0 for i in range(half)]
    else:
        for a, n in enumerate(sections):
            axes += [a] * n
    for i in range(half):
        w = positions[axes[i]].double() * float(inv_freq[i])
        c, s = w.cos()[:, None], w.sin()[:, None]
        a, b = x[..., i].double(), x[..., i + half].double()
        y[..., i], y[..., i + half] = a * c - b * s, b * c + a * s
        size[..., i] = size[..., i + half] = a.abs() + b.abs()
    return y, size


def tables(P, num_pages, start, new, free, table, max_rows, slots, positions):
    """The results of nk_step_tables as numpy arrays (one sequence, row and page at a time)."""
    table, slots, positions = table.copy(), slots.copy(), positions.copy()
    cu, ctx, k = [0], [], 0
    for b, (s, n) in enumerate(zip(start, new)):
        ok = s >= 0 and n >= 0 and s + n <= table.shape[1] * P
        rows = max(n, 0)
        ctx.append(s + n if ok else 0)
        if ok:
            for pi in range(-(-s // P), -(-(s + n) // P)):
                page = int(free[k]) if k < len(free) else -1
                table[b, pi] = page if 0 <= page < num_pages else -1
                k += 1
        for t in range(rows):
            j = cu[-1] + t
            if j >= max_rows:
                break
            page = int(table[b, (s + t) // P]) if ok else -1
            slots[j] = page * P + (s + t) % P if 0 <= page < num_pages else -1
            positions[j] = s + t if ok else -1
        cu.append(cu[-1] + rows)
    return table, np.array(cu), np.array(ctx), slots, positions, k
