"""Paged attention at the ends of an 8-bit cache's scales, against float64."""
from __future__ import annotations

import pytest
import torch

import cache_reference as ref
from test_gpu_attention_paths import widened
from test_gpu_paged_attention import dev, make_table, rng  # noqa: F401

pytestmark = pytest.mark.gpu

LENGTHS = [300, 1, 0, 37, 3000]


def f32(x):
    return float(torch.tensor(x, dtype=torch.float32))


def setup(dev, Hkv, D, k_std, v_std, q_std, wide):  # noqa: F811
    """q, k, v, table, lengths: one key head joins four warps of a block, four have one each; wide tables go to runs."""
    g = rng(dev, Hkv + D)
    table, pages = make_table(LENGTHS, 16, dev, g)
    table = widened(table, 16, 300000) if wide else table
    code = lambda std: (std * torch.randn((pages, 16, Hkv, D), generator=g, device=dev)).clamp(-448, 448).to(torch.float8_e4m3fn)   # noqa: E731
    q = (torch.randn((len(LENGTHS), 4 * Hkv, D), generator=g, device=dev).clamp(-1.9, 1.9) * q_std).to(torch.bfloat16)
    return q, code(k_std), code(v_std), table, torch.tensor(LENGTHS, dtype=torch.int32, device=dev)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("Hkv,D", [(1, 64), (4, 128), (2, 256)])
@pytest.mark.parametrize("v_scale,v_std", [(2.0 ** -126, 60.0), (1.3e-38, 60.0), (2.0 ** -112, 1.0), (3e30, 60.0), (2.0 ** 126, 0.25)])
def test_value_scales(dev, wide, Hkv, D, v_scale, v_std):  # noqa: F811
    from memory_bound_moe_gb300 import KVCache, moe_paged_attention
    q, k, v, table, n = setup(dev, Hkv, D, 40.0, v_std, 1.0, wide)
    want, want_lse, tol, ltol = ref.attention(q, k, v, table, n, D ** -0.5, 0, 0.021, 1.0)
    cache = KVCache(k, v, 0.021, v_scale)
    lse = torch.empty_like(want_lse, dtype=torch.float32)
    out = moe_paged_attention(q, cache, table, n, lse=lse)
    # a result below 2^-126 is off by half a step of the subnormals, 2^-134
    off = (out.double() / f32(v_scale) - want).abs()
    assert (off <= tol + 2.0 ** -134 / v_scale).all(), float((off / (tol + 2.0 ** -134 / v_scale)).max())
    there = want_lse.isfinite()
    assert ((lse.double() - want_lse).abs()[there] <= ltol[there]).all()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("Hkv,D", [(1, 64), (4, 128), (2, 256)])
@pytest.mark.parametrize("k_scale,scale,k_std,q_std", [
    (2.0 ** 126, 8.0, 2.0 ** -6, 2.0 ** -124),              # scale times k_scale is above float32's range, the scores are not
    (2.0 ** 126, -1.5 * 2.0 ** 8, 2.0 ** -6, 2.0 ** -126),
    (2.0 ** 100, 2.0 ** 100, 2.0 ** -8, 0.0),               # all scores 0
    (2.0 ** 126, 2.0 ** -128, 40.0, 0.5),
    (2.0 ** -126, 1.37 * 2.0 ** -12, 100.0, 2.0 ** 126),    # and here below it
    (2.0 ** -126, 2.0 ** 100, 40.0, 2.0 ** 18),
    (2.0 ** -126, 3e38, 40.0, 2.0 ** -5)])
def test_key_scales(dev, wide, Hkv, D, k_scale, scale, k_std, q_std):  # noqa: F811
    from memory_bound_moe_gb300 import KVCache, moe_paged_attention
    q, k, v, table, n = setup(dev, Hkv, D, k_std, 60.0, q_std, wide)
    want, want_lse, tol, ltol = ref.attention(q, k, v, table, n, f32(scale), 0, f32(k_scale), 0.017)
    assert want.isfinite().all()
    lse = torch.empty_like(want_lse, dtype=torch.float32)
    out = moe_paged_attention(q, KVCache(k, v, k_scale, 0.017), table, n, scale=scale, lse=lse)
    assert ((out.double() - want).abs() <= tol).all()
    there = want_lse.isfinite()
    assert ((lse.double() - want_lse).abs()[there] <= ltol[there]).all()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("scale", [3.4e38, -3.4e38, 1e-44])
def test_scales_of_a_bfloat16_cache(dev, wide, scale):  # noqa: F811
    """The scale times log2 e is above float32's range; q makes the scores ordinary ones."""
    from memory_bound_moe_gb300 import KVCache, moe_paged_attention
    q, k, v, table, n = setup(dev, 2, 64, 0.25, 1.0, 2.0 ** -126 if abs(scale) > 1 else 2.0 ** 120, wide)
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    want, want_lse, tol, ltol = ref.attention(q, k, v, table, n, f32(scale))
    lse = torch.empty_like(want_lse, dtype=torch.float32)
    out = moe_paged_attention(q, KVCache(k, v), table, n, scale=scale, lse=lse)
    assert ((out.double() - want).abs() <= tol).all()
    there = want_lse.isfinite()
    assert ((lse.double() - want_lse).abs()[there] <= ltol[there]).all()
