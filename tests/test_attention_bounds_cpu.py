"""That the long sequences' bounds see a few tokens left out or taken twice (the mistake is made in the reference)."""
from __future__ import annotations

import pytest
import torch

import attention_bounds as bounds

SMS = 152


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,D,lost", [(40000, 64, 64), (40000, 128, 64), (70000, 64, 128), (70000, 64, 64)])
def test_random_sequences_show_a_lost_tile(kind, n, D, lost):
    g = torch.Generator().manual_seed(n + D)
    dt = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
    q = (0.1 * torch.randn((1, 4, D), generator=g)).to(torch.bfloat16)   # scores well below 1: their errors count little
    k, v = (torch.randn((-(-n // 16), 16, 1, D), generator=g).to(dt) for _ in "kv")
    table = torch.arange(k.shape[0], dtype=torch.int32)[None]
    chain = bounds.chain([n], 1, 4, SMS)
    call = lambda **kw: bounds.attention(q, k, v, table, [n], D ** -0.5, chain, **kw)   # noqa: E731
    want, want_lse, tol, ltol = call()
    assert (tol < 0.02 * v.float().abs().max()).all()
    for first in (0, 20000, n - lost):
        out, lse, _, _ = call(without=[(first, first + lost)])
        # a mistaken kernel's result is rounded, and may be off by the bound besides: twice the bound shows
        assert ((out - want).abs() > 2 * tol).any(-1).all()
        assert ((lse - want_lse).abs() > 2 * ltol).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,D", [(1000003, 64), (1000003, 256), (131072, 64), (70001, 128), (40000, 128), (9000, 256), (777, 64)])
def test_counted_sequences_show_16_tokens(e4m3, n, D):
    chain = bounds.chain([n], 1, 4, SMS)
    R = bounds.passes(n, D)
    for times in (0, 2):
        for first in (0, 16, n // 3, n - 16):
            taken = torch.ones(n, dtype=torch.float64)
            taken[first:first + 16] = times
            seen = 0
            for r in range(R):
                cols = bounds.column(n, D, R, r, 1, "cpu")
                mean = bounds.counted(cols, D) / n
                wrong = (bounds.counted(cols, D, taken) / taken.sum()).to(torch.bfloat16).double()
                tol = bounds.counted_tol(mean, chain, e4m3)
                seen += int(((wrong - mean).abs() > tol).sum())
                # and the right means, rounded, are within it
                assert ((mean.to(torch.bfloat16).double() - mean).abs() <= tol).all()
            assert seen > 0, (times, first)
    if not e4m3:
        assert bounds.counted_lse_tol(n, chain, False) < 16 / n
