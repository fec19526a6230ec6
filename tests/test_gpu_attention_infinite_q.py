"""Paged attention of queries that hold infinities: scores of -infinity alone
are an empty softmax, any other infinite score makes the row NaN."""
from __future__ import annotations

import math

import pytest
import torch

from test_gpu_attention_paths import widened
from test_gpu_paged_attention import KINDS, dev, make_table, rng  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("size", [1.0, 3e5, 1e30])
def test_infinite_queries(dev, kind, wide, size):  # noqa: F811
    """Column 0 of q is -infinity, +infinity or ordinary and the keys' column 0 positive; the rest is of `size`."""
    from memory_bound_moe_gb300 import KVCache, moe_paged_attention
    g = rng(dev, 3)
    lengths = [300, 17, 0, 2000]
    table, pages = make_table(lengths, 16, dev, g)
    table = widened(table, 16, 300000) if wide else table
    k, v = (torch.randn((pages, 16, 2, 64), generator=g, device=dev) for _ in "kv")
    k[..., 0] = k[..., 0].abs() + 0.5
    t = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
    q = size * torch.randn((4, 6, 64), generator=g, device=dev)
    q[:, 0, 0], q[:, 1, 0], q[:, 5, 0] = -math.inf, math.inf, -math.inf
    lse = torch.empty((4, 6), device=dev)
    out = moe_paged_attention(q.to(torch.bfloat16), KVCache(k.to(t), v.to(t)), table,
                              torch.tensor(lengths, dtype=torch.int32, device=dev), scale=0.125 / size, lse=lse)
    there = [0, 1, 3]
    for h in (0, 5):
        assert (out[:, h] == 0).all() and (lse[:, h] == -math.inf).all()
    assert out[there, 1].isnan().all() and lse[there, 1].isnan().all()
    assert out[:, 2:5].isfinite().all() and lse[there, 2:5].isfinite().all()
    assert (out[2] == 0).all() and (lse[2] == -math.inf).all()
