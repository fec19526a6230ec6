"""Paged attention where values cancel to far below their size, so that the
rounding of the softmax's weights shows in front of the output's own."""
from __future__ import annotations

import pytest
import torch

import attention_bounds as bounds
from test_gpu_attention_paths import widened
from test_gpu_paged_attention import KINDS, dev, make_table, rng  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (12, 1), (8, 4)])
def test_values_that_cancel(dev, kind, wide, D, Hq, Hkv):  # noqa: F811
    """Values of one size and alternating sign at tokens whose weights differ by up to 3%."""
    from memory_bound_moe_gb300 import KVCache, moe_paged_attention
    g = rng(dev, D + Hq)
    lengths = [2, 4, 16, 64, 2, 2, 4, 6]
    table, pages = make_table(lengths, 16, dev, g)
    table = widened(table, 16, 300000) if wide else table
    t, k_scale, v_scale = (torch.bfloat16, 1.0, 1.0) if kind == "bf16" else (torch.float8_e4m3fn, 2.0 ** -14, 0.017)
    k = torch.zeros((pages, 16, Hkv, D), device=dev)
    k[..., 0] = (448 * (2 * torch.rand((pages, 16, Hkv), generator=g, device=dev) - 1)).to(torch.float8_e4m3fn).float()
    k[..., 0] *= 2.0 ** -14 / k_scale
    v = torch.where(torch.arange(16, device=dev) % 2 == 0, 1.0, -1.0)[None, :, None, None] * torch.ones((pages, 16, Hkv, D), device=dev)
    v *= 448 if kind == "e4m3" else 1
    k, v = k.to(t), v.to(t)
    q = torch.zeros((len(lengths), Hq, D), device=dev)
    q[..., 0] = 0.3 + torch.rand((len(lengths), Hq), generator=g, device=dev)
    q = q.to(torch.bfloat16)
    n = torch.tensor(lengths, dtype=torch.int32, device=dev)
    f32 = float(torch.tensor(v_scale, dtype=torch.float32))
    want, want_lse, tol, ltol = bounds.attention(q, k, v, table, n, 1.0, 64, k_scale=k_scale, v_scale=f32, joined=16)
    assert (want.abs() < 0.05 * float(v.float().abs().max()) * f32).all()
    lse = torch.empty((len(lengths), Hq), device=dev)
    out = moe_paged_attention(q, KVCache(k, v, k_scale, v_scale), table, n, scale=1.0, lse=lse)
    off = (out.double() - want).abs() / tol
    assert (off <= 1).all(), f"{float(off.max()):.3g} of the bound"
    assert ((lse.double() - want_lse).abs() <= ltol).all()
