"""The paged cache's operators in float64 and whole numbers, written from their
definitions, and bounds of the library's rounding errors.

Half a step of a type relative to a value: bfloat16 2^-8, f16 2^-11, E4M3 2^-4
(2^-10 absolute below 2^-6), float32 2^-24. The tensor cores' float32 sums are
taken as one truncation, 2^-23, per term.
"""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -23


def attention(q, k_cache, v_cache, table, lengths, scale, window=0, k_scale=1.0, v_scale=1.0):
    """(out, lse, bound of out's error, bound of lse's), float64, on q's device."""
    B, Hq, D = q.shape
    pages, P, Hkv, _ = k_cache.shape
    G = Hq // Hkv
    f64 = dict(dtype=torch.float64, device=q.device)
    out, lse = torch.zeros((B, Hq, D), **f64), torch.full((B, Hq), -math.inf, **f64)
    tol, ltol = torch.zeros((B, Hq, D), **f64), torch.zeros((B, Hq), **f64)
    e4m3 = k_cache.dtype == torch.float8_e4m3fn
    for b in range(B):
        n = min(max(int(lengths[b]), 0), table.shape[1] * P)
        at = torch.arange(max(0, n - window) if window else 0, n, device=q.device)
        page = table[b].long()[at // P]
        ok = (page >= 0) & (page < pages)
        at, page = at[ok], page[ok]
        if at.numel() == 0:
            continue
        k, v = (c[page, at % P].double().transpose(0, 1) for c in (k_cache, v_cache))   # [Hkv, n, D]
        x = q[b].double().view(Hkv, G, D)
        s = scale * k_scale * (x @ k.transpose(1, 2))                                   # [Hkv, G, n]
        size = abs(scale) * k_scale * (x.abs() @ k.abs().transpose(1, 2)).amax(-1, keepdim=True)
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        total = p.sum(-1, keepdim=True)
        y = (p @ v) / total * v_scale
        mass = (p @ v.abs()) / total * v_scale
        # scores: D terms, the factor and the distance to the maximum; q of an E4M3 cache is exact but for
        # values 2^-31 below the row's largest. Weights: the exponential (2^-21) and their rounding.
        dx = size * (D + 16) * U32
        dw = torch.expm1(2 * dx) + 2.0 ** -21 + (2.0 ** -11 if e4m3 else 2.0 ** -16) + (at.numel() + 64) * U32
        out[b], lse[b] = y.view(Hq, D), (m + torch.log(total)).view(Hq)
        tol[b] = (2.0 ** -8 * y.abs() + 2 * dw * mass + 1e-38).view(Hq, D)
        ltol[b] = (2 * dx + 2.0 ** -21 + (at.numel() + 64) * U32 + 4 * U32 * (m.abs() + 16)).view(Hq)
    return out, lse, tol, ltol


def page_table(cached, added, table, free_pages, free_count, P, N):
    """Lists in, lists out, one token at a time; `table` (a list of rows) is changed in place."""
    M = len(table[0]) if table else 0
    free = min(max(free_count, 0), len(free_pages))
    lengths, starts, positions, slots, refused = [], [0], [0] * N, [-1] * N, 0
    taken = given = 0
    for b, (c, a) in enumerate(zip(cached, added)):
        c, a = max(c, 0), max(a, 0)
        have, need = -(-c // P), -(-(c + a) // P)
        start = starts[-1]
        starts.append(start + a)
        ok = need <= M and start + a <= N
        if ok and need > have:
            taken += need - have
            ok = taken <= free
            if ok:
                given = taken
        lengths.append(c + a if ok else c)
        refused += not ok
        if not ok:
            continue
        for j in range(have, need):
            table[b][j] = free_pages[free - 1 - (taken - (need - have) + j - have)]
        for i in range(a):
            pos = c + i
            positions[start + i] = pos
            if table[b][pos // P] >= 0:
                slots[start + i] = table[b][pos // P] * P + pos % P
    return lengths, starts, positions, slots, free - given, refused


def rotate(x, cos_sin, positions, interleaved):
    """x [N, heads, D] in float64, rotated; and the bound of a float32 evaluation's error."""
    rot = cos_sin.shape[1]
    cs = cos_sin.double()[positions.long()]
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    x = x.double()
    y, size = x.clone(), torch.zeros_like(x)
    ia = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    ib = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = (a * c).abs() + (b * s).abs()
    size[..., ib] = (b * c).abs() + (a * s).abs()
    return y, 2 * 2.0 ** -24 * size


def cached_values(x, err, scale, e4m3):
    """What the cache holds for float64 values x known to err, and the bound of its error."""
    if not e4m3:
        return x, err + 2.0 ** -8 * (x.abs() + err)
    y = (x / scale).clamp(-448, 448)
    e = err / scale + 2 * 2.0 ** -24 * (x / scale).abs()   # 1 / scale and the product are rounded
    return y, e + torch.maximum(2.0 ** -4 * (y.abs() + e), torch.full_like(y, 2.0 ** -10))
