"""The 4-bit layer rounds to bfloat16 once: its activation is held in float32
and enters fc2 with the 11 bits of f16.

Every output is 1.5 times one activation here, so both roundings show: the
error is at most half a step of the output, 2^-11 of the activation, and what
the float32 sums of few_reference.py's bounds lose in front of them."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from few_reference import BLOCK, fsum, random_fp4, weights64
from test_gpu_layer import dev  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T", [1, 7, 12, 32])
def test_one_rounding(dev, T, fmt):  # noqa: F811
    from memory_bound_moe_gb300 import moe_layer_fp4
    H, I = 256, 64
    rng = np.random.default_rng(71)
    c13, s13 = random_fp4(rng, (1, 2 * I, H), fmt)
    g13 = 1000.0 if fmt == "nvfp4" else 1.0
    codes = np.zeros((1, H, I), dtype=np.uint8)
    codes[0, np.arange(H), np.arange(H) % I] = 3                          # 1.5
    c2 = codes[..., 0::2] | (codes[..., 1::2] << 4)
    s2 = np.full((1, H, I // BLOCK[fmt]), 0x38 if fmt == "nvfp4" else 127, dtype=np.uint8)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    g = (torch.full((1,), g13, device=dev), torch.ones(1, device=dev)) if fmt == "nvfp4" else (None, None)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16)
    out = moe_layer_fp4(torch.zeros((T, 1), device=dev), x.to(dev), up(c13), up(s13), up(c2), up(s2), 1, True, fmt, *g)
    w = weights64(c13[0], s13[0], fmt, g13)
    xd = x.double().numpy()
    gate, u = xd @ w[:I].T, xd @ w[I:].T
    dg, du = fsum(H) * (np.abs(xd) @ np.abs(w[:I]).T), fsum(H) * (np.abs(xd) @ np.abs(w[I:]).T)
    sg = gate / (1 + np.exp(-gate))
    a = sg * u
    # |silu'| <= 1.1; the exponential, quotient, products and scales: 2^-19
    da = 1.1 * dg * np.abs(u) + (np.abs(sg) + 1.1 * dg) * du + (2.0 ** -11 + 2.0 ** -19) * np.abs(a)
    pick = np.arange(H) % I
    ref, d = 1.5 * a[:, pick], 1.5 * da[:, pick]
    half = 2.0 ** (np.floor(np.log2(np.abs(ref) + d)) - 8)
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= d + half).all(), (int((err > d + half).sum()), float((err / (d + half)).max()))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T", [1, 7, 20])
def test_activations_of_very_different_size(dev, T, fmt):  # noqa: F811
    """Columns down to 2^-48 (MXFP4) of their neighbours, in groups of 8: each
    keeps 11 bits down to 2^-28 of the largest that fc2 takes with it (32 of every
    128 columns of a chunk of 512), and loses at most 2^-38 of that below."""
    from memory_bound_moe_gb300 import moe_layer_fp4
    H = I = 512
    rng = np.random.default_rng(72)
    c13, s13 = random_fp4(rng, (1, 2 * I, H), fmt)
    c13 |= 0x11                                                           # no zero weights
    steps = np.array([0x38, 0x30, 0x20, 0x10, 0x08, 0x01] if fmt == "nvfp4" else [122, 118, 114, 108, 102, 98])
    size = steps[rng.integers(0, 6, I // 8)].repeat(8).astype(np.uint8)   # of 8 neighbouring columns
    size[96:128], size[224:256] = steps[5], steps[5]                      # a run without any large one
    s13[0, :I], s13[0, I:] = size[:, None], size[:, None]
    g13 = 20.0 if fmt == "nvfp4" else 1.0
    codes = np.zeros((1, H, I), dtype=np.uint8)
    codes[0, np.arange(H), np.arange(I)] = 3                              # 1.5
    c2 = codes[..., 0::2] | (codes[..., 1::2] << 4)
    s2 = np.full((1, H, I // BLOCK[fmt]), 0x38 if fmt == "nvfp4" else 127, dtype=np.uint8)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    g = (torch.full((1,), g13, device=dev), torch.ones(1, device=dev)) if fmt == "nvfp4" else (None, None)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16)
    out = moe_layer_fp4(torch.zeros((T, 1), device=dev), x.to(dev), up(c13), up(s13), up(c2), up(s2), 1, True, fmt, *g)
    w = weights64(c13[0], s13[0], fmt, g13)
    xd = x.double().numpy()
    gate, u = xd @ w[:I].T, xd @ w[I:].T
    dg, du = fsum(H) * (np.abs(xd) @ np.abs(w[:I]).T), fsum(H) * (np.abs(xd) @ np.abs(w[I:]).T)
    sg = gate / (1 + np.exp(-gate))
    a = sg * u
    assert np.abs(a).min() < 2.0 ** -20 * np.abs(a).max()
    most = np.abs(a).reshape(T, 4, 4, 32).max((1, 3), keepdims=True)      # [run of 128][32 columns of each run]
    most = np.broadcast_to(most, (T, 4, 4, 32)).reshape(T, I)
    da = 1.1 * dg * np.abs(u) + (np.abs(sg) + 1.1 * dg) * du + (2.0 ** -11 + 2.0 ** -19) * np.abs(a) + 2.0 ** -38 * most
    ref, d = 1.5 * a, 1.5 * da
    half = 2.0 ** (np.floor(np.log2(np.abs(ref) + d)) - 8)
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= d + half).all(), (int((err > d + half).sum()), float((err / (d + half)).max()))
