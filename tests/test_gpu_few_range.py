"""Products with 4-bit weights at the ends of the number range: very small and
very large factors and tensor scales, and the border of what x keeps."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from few_reference import BLOCK, check_gemv, weights64
from test_gpu_gemv_fp4 import FMTS, make
from test_gpu_layer import Layer, dev, run_and_check, tokens  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 4, 20])
@pytest.mark.parametrize("ex,scale", [(-64, 67), (-100, 97), (-40, 40), (100, 34), (60, 60), (20, 200)])
def test_mxfp4_factors_beyond_one_float(dev, T, ex, scale):  # noqa: F811
    """x about 2^ex and weights about 2^(scale - 127): results that float32
    holds, also where the powers of two behind x and behind the weights have a
    product that it does not."""
    from memory_bound_moe_gb300 import moe_gemv_fp4
    N, K = 40, 1120
    x, codes, scales, cd, _ = make(T, N, K, "mxfp4", dev, 51)
    scales[:] = scale
    x = (x.float() * 2.0 ** ex).to(torch.bfloat16)
    y = moe_gemv_fp4(x, cd, torch.from_numpy(scales).to(dev), "mxfp4", out_dtype=torch.float32)
    check_gemv(y, x, weights64(codes, scales, "mxfp4"), f"2^{ex}, scale {scale}")
    # tokens of ordinary size beside them
    if T > 1:
        x[0] *= 2.0 ** -ex
        y = moe_gemv_fp4(x, cd, torch.from_numpy(scales).to(dev), "mxfp4", out_dtype=torch.float32)
        check_gemv(y, x, weights64(codes, scales, "mxfp4"), f"beside 2^{ex}, scale {scale}")


@pytest.mark.parametrize("T", [2, 12])
@pytest.mark.parametrize("ex", [40, 100, 127])
def test_mxfp4_zero_weights_with_the_largest_scales(dev, T, ex):  # noqa: F811
    """Blocks of zeros may have any finite scale byte; x large."""
    from memory_bound_moe_gb300 import moe_gemv_fp4
    N, K = 33, 1056
    x = torch.full((T, K), 2.0 ** ex, dtype=torch.bfloat16, device=dev)
    codes = torch.zeros((N, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.full((N, K // 32), 254, dtype=torch.uint8, device=dev)
    assert (moe_gemv_fp4(x, codes, scales, "mxfp4", out_dtype=torch.float32) == 0).all()


@pytest.mark.parametrize("T", [1, 9])
@pytest.mark.parametrize("g", [2e-39, 1e-44, 2.0 ** -126, 3e38])
def test_nvfp4_every_allowed_tensor_scale(dev, T, g):  # noqa: F811
    """Tensor scales whose reciprocal is no float32, or a subnormal one."""
    from memory_bound_moe_gb300 import moe_gemv_fp4
    g = float(np.float32(g))
    N, K = 40, 288
    x, codes, scales, cd, sd = make(T, N, K, "nvfp4", dev, 52)
    codes[7] = 0
    cd = torch.from_numpy(codes).to(dev)
    x = (x.float() * (2.0 ** -60 if g < 1 else 2.0 ** 60)).to(torch.bfloat16)
    y = moe_gemv_fp4(x, cd, sd, "nvfp4", g, out_dtype=torch.float32)
    check_gemv(y, x, weights64(codes, scales, "nvfp4", g), f"g = {g}")


@pytest.mark.parametrize("T", [2, 12])
@pytest.mark.parametrize("g13,g2", [(2e-39, 1e30), (3e-42, 1e35), (3e38, 2.0 ** -126)])
def test_layer_nvfp4_extreme_tensor_scales(dev, T, g13, g2):  # noqa: F811
    """Weights and x so far apart that the sums before the division by the
    tensor scale, or its reciprocal, lie at an end of float32."""
    E, H, I, k = 4, 96, 64, 2
    layer = Layer(E, H, I, "nvfp4", dev, 53)
    layer.g = [np.full(E, g13, np.float32), np.full(E, g2, np.float32)]
    layer.gd = [torch.from_numpy(g).to(dev) for g in layer.g]
    logits, x = tokens(T, E, H, dev, 54)
    x = (x.float() * (2.0 ** -120 if g13 < 1 else 2.0 ** 100)).to(torch.bfloat16)
    run_and_check(layer, logits, x, k, True, f"g = {g13}, {g2}")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("big", [1.0, 1.9921875])
def test_what_x_keeps_beside_a_large_value(dev, fmt, big):  # noqa: F811
    """Beside `big`, a value down to 2^-31 of it keeps all its bits; one
    smaller loses at most 2^-39 of it."""
    from memory_bound_moe_gb300 import moe_gemv_fp4
    K = 128
    one = 0x38 if fmt == "nvfp4" else 127
    scales = torch.full((1, K // BLOCK[fmt]), one, dtype=torch.uint8, device=dev)
    codes = torch.zeros((1, K // 2), dtype=torch.uint8, device=dev)
    codes[0, 5] = 0x20                                          # weight 11 is 1, weight 100 is 0
    for e in (-20, -30, -31, -32, -33, -36, -40):
        for m in (1.0, 1.0078125, 1.5, 1.9921875):              # 8 significant bits
            x = torch.zeros((1, K), dtype=torch.bfloat16)
            x[0, 100], x[0, 11] = big, m * 2.0 ** e
            y = float(moe_gemv_fp4(x.to(dev), codes, scales, fmt, out_dtype=torch.float32))
            if m * 2.0 ** e >= big * 2.0 ** -31:
                assert y == float(x[0, 11]), (e, m)
            assert abs(y - float(x[0, 11])) <= big * 2.0 ** -39, (e, m)
