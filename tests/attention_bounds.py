"""Paged attention in float64 with bounds of the library's errors that do not
grow with the sequence but with what one warp adds up.

A product's float32 sums are taken as one truncation, 2^-23, per term. A warp
adds up at most ``chain`` tokens of a sequence, and up to ``joined`` partial
results are added behind it.
"""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -23
JOINED = 96     # partial results that a sum may pass through: those of 640 runs over eight warps, and these


def chain(lengths, Hkv, G, sms):
    """Tokens of a sequence that one warp adds up, at most. Short ones (up to 16640 tokens) may go to clusters of up
    to 8 blocks, whose four warps share up to 2080 tokens; else all heads' tokens, and a few tiles of at most 128
    tokens for each unit, are shared evenly by a block per SM or more, whose warps have each a head, or a quarter
    of the tokens."""
    units = Hkv * -(-G // 16) / 4
    runs = math.ceil(sum(units * (n + 512) for n in lengths) / sms) + 128
    longest = max(lengths)
    return max(runs, min(longest, 2080) // 4 + 128 if longest <= 8 * 2080 else 0)


def attention(q, k_cache, v_cache, table, lengths, scale, chain, window=0, k_scale=1.0, v_scale=1.0, without=(), joined=JOINED):
    """(out, lse, bound of out's error, bound of lse's), float64, on q's device. ``without``: (first, last + 1)
    of tokens that are left out in every sequence, for tests of the bounds."""
    B, Hq, D = q.shape
    pages, P, Hkv, _ = k_cache.shape
    G = Hq // Hkv
    f64 = dict(dtype=torch.float64, device=q.device)
    out, lse = torch.zeros((B, Hq, D), **f64), torch.full((B, Hq), -math.inf, **f64)
    tol, ltol = torch.zeros((B, Hq, D), **f64), torch.zeros((B, Hq), **f64)
    e4m3 = k_cache.dtype == torch.float8_e4m3fn
    sums = (chain + joined) * U32
    for b in range(B):
        n = min(max(int(lengths[b]), 0), table.shape[1] * P)
        at = torch.arange(max(0, n - window) if window else 0, n, device=q.device)
        for lo, hi in without:
            at = at[(at < lo) | (at >= hi)]
        page = table[b].long()[at // P]
        ok = (page >= 0) & (page < pages)
        at, page = at[ok], page[ok]
        if at.numel() == 0:
            continue
        for h in range(Hkv):
            k, v = (c[page, at % P, h].double() for c in (k_cache, v_cache))     # [n, D]
            x = q[b, h * G:(h + 1) * G].double()
            s = scale * k_scale * (x @ k.T)                                       # [G, n]
            size = abs(scale) * k_scale * (x.abs() @ k.abs().T).amax(-1, keepdim=True)
            m = s.amax(-1, keepdim=True)
            p = torch.exp(s - m)
            total = p.sum(-1, keepdim=True)
            y, mass = (p @ v) / total * v_scale, (p @ v.abs()) / total * v_scale
            # a score: D products, the factor, the distance to the largest
            dx = size * (D + 16) * U32
            # a weight: the exponential and its rounding, with an 8-bit cache to 2^-22, or 2^-40 of the
            # largest, else to 2^-16
            dw = torch.expm1(2 * dx) + 2.0 ** -21 + (2.0 ** -22 if e4m3 else 2.0 ** -16)
            small = (2.0 ** -40 * v.abs().sum(0) / total * v_scale) if e4m3 else 0.0
            heads = slice(h * G, (h + 1) * G)
            out[b, heads], lse[b, heads] = y, (m + torch.log(total))[:, 0]
            tol[b, heads] = 2.0 ** -8 * y.abs() + (2 * dw + sums) * mass + sums * y.abs() + small + 2.0 ** -133
            # the largest score and the sum's logarithm are float32 in units of ln 2; with an 8-bit cache 15 apart
            ltol[b, heads] = (2 * dx + 2.0 ** -21 + sums + 2.0 ** -22 * (m.abs() + torch.log(total) + 24))[:, 0]
    return out, lse, tol, ltol


# Sequences whose scores are all 0, so that the output counts tokens: the value of a token is 1 in one column, 0 in
# the others. A sequence is cut into equal blocks, a column (of one of several passes) each; a block holds at most
# 1024 tokens, so that 16 tokens left out or taken twice are more than a bfloat16's rounding.

COUNTED = 1024


def passes(n, D):
    return max(1, -(-n // (COUNTED * D)))


def column(n, D, count, r, head, device):
    """For each of n tokens the column that it counts in during pass r of `count`, or -1."""
    block = torch.arange(n, device=device) * (D * count) // max(1, n)
    return torch.where(block // D == r, (block % D + 7 * head) % D, -1)


def counted(cols, D, times=None):
    """The tokens that each column counts; `times`: how often each token is taken (default once)."""
    there = cols >= 0
    w = torch.ones(cols.shape, dtype=torch.float64, device=cols.device) if times is None else times.double()
    return torch.zeros(D, dtype=torch.float64, device=cols.device).index_add_(0, cols[there], w[there])


def counted_tol(mean, chain, e4m3):
    """Bound of the error of a column's mean. The weights are 1 (2^15 with an 8-bit cache, to 2^-22), and the second
    bfloat16 term at most adds 2^-20."""
    return (2.0 ** -8 + 2.0 ** -20 + (2 * (chain + JOINED) * U32 + 2.0 ** -21 if e4m3 else 0.0)) * mean


def counted_lse_tol(n, chain, e4m3):
    """Bound of the error of ln n: the sum of the ones is exact, with an 8-bit cache a lane adds up a quarter of
    what its warp does, rounded to nearest."""
    return 2.0 ** -22 * (math.log(n) + 24) + (((chain / 4 + JOINED) * 2.0 ** -24 + 2.0 ** -22) if e4m3 else 0.0)
