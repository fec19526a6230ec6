"""moe_gemv_fp4 on the GPU against float64 (bounds: few_reference.py)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from few_reference import BLOCK, check_gemv, random_fp4, weights64

pytestmark = pytest.mark.gpu
FMTS = ["nvfp4", "mxfp4"]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from memory_bound_moe_gb300 import build
    build.build()
    return torch.device("cuda:0")


def make(T, N, K, fmt, dev, seed, spread=3):
    rng = np.random.default_rng(seed)
    codes, scales = random_fp4(rng, (N, K), fmt, spread)
    x = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).to(torch.bfloat16).to(dev)
    return x, codes, scales, torch.from_numpy(codes).to(dev), torch.from_numpy(scales).to(dev)


SHAPES = [(1, 1, 32), (1, 16, 64), (3, 17, 96), (8, 33, 160), (9, 100, 2880), (16, 257, 768), (17, 64, 7168),
          (31, 1000, 352), (32, 512, 2048), (1, 4096, 7168), (5, 5760, 2880), (2, 15, 32768), (1, 20011, 64)]


@pytest.mark.parametrize("T,N,K", SHAPES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_against_float64(dev, T, N, K, fmt, dtype):
    from memory_bound_moe_gb300 import moe_gemv_fp4
    x, codes, scales, cd, sd = make(T, N, K, fmt, dev, T + N + K)
    g = 37.5 if fmt == "nvfp4" else 1.0
    y = moe_gemv_fp4(x, cd, sd, fmt, g, out_dtype=dtype)
    check_gemv(y, x, weights64(codes, scales, fmt, g), f"T={T} N={N} K={K} {fmt}")
    assert torch.equal(y, moe_gemv_fp4(x, cd, sd, fmt, g, out_dtype=dtype))   # the same bits again


@pytest.mark.parametrize("fmt", FMTS)
def test_every_code_and_scale_is_exact(dev, fmt):
    """One weight per output: a unit x picks it, so the product is the weight's
    value itself, exact in float32."""
    from memory_bound_moe_gb300 import moe_gemv_fp4
    K, b = 32, BLOCK[fmt]
    bytes_ = np.arange(256) if fmt == "nvfp4" else np.arange(0, 253)   # MXFP4: 6 * 2^125 is finite
    for k0 in (0, 7, 31):
        for code in range(16):
            N = len(bytes_)
            codes = np.zeros((N, K // 2), dtype=np.uint8)
            codes[:, k0 // 2] = code << (4 * (k0 % 2))
            scales = np.repeat(bytes_.astype(np.uint8)[:, None], K // b, 1)
            x = torch.zeros((2, K), dtype=torch.bfloat16)
            x[1, k0] = 1
            y = moe_gemv_fp4(x.to(dev), torch.from_numpy(codes).to(dev), torch.from_numpy(scales).to(dev), fmt, 1.0,
                             out_dtype=torch.float32).cpu().numpy()
            want = weights64(codes, scales, fmt)[:, k0].astype(np.float32)
            nan = np.isnan(want)
            assert np.array_equal(y[1][~nan], want[~nan]), (code, k0, np.argwhere(y[1] != want)[:4])
            assert np.isnan(y[1][nan]).all()


@pytest.mark.parametrize("spread", [0, 20, 40, 90])
def test_mxfp4_scales_far_apart(dev, spread):
    """Blocks of a row up to 2^180 apart: each keeps its own size."""
    from memory_bound_moe_gb300 import moe_gemv_fp4
    T, N, K = 4, 70, 1024
    x, codes, scales, cd, sd = make(T, N, K, "mxfp4", dev, 5 + spread, spread)
    y = moe_gemv_fp4(x, cd, sd, "mxfp4", out_dtype=torch.float32)
    check_gemv(y, x, weights64(codes, scales, "mxfp4"), f"spread {spread}")
    # rows of one size each, far from their neighbours in the same tile
    scales[:] = (127 + (np.arange(N) % 16 - 8) * (spread // 8))[:, None]
    y = moe_gemv_fp4(x, cd, torch.from_numpy(scales).to(dev), "mxfp4", out_dtype=torch.float32)
    check_gemv(y, x, weights64(codes, scales, "mxfp4"), f"rows {spread}")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [1, 5, 20])
def test_tokens_of_very_different_size(dev, fmt, T):
    """Each token keeps the precision of its own size, whatever its batch."""
    from memory_bound_moe_gb300 import moe_gemv_fp4
    N, K = 48, 2880
    x, codes, scales, cd, sd = make(T, N, K, fmt, dev, 77)
    x *= torch.pow(2.0, torch.linspace(-60, 60, T, device=dev))[:, None].to(torch.bfloat16)
    y = moe_gemv_fp4(x, cd, sd, fmt, 1.0, out_dtype=torch.float32)
    w = weights64(codes, scales, fmt)
    check_gemv(y, x, w, "sizes")
    for t in range(T):
        alone = moe_gemv_fp4(x[t:t + 1].contiguous(), cd, sd, fmt, 1.0, out_dtype=torch.float32)
        check_gemv(alone, x[t:t + 1], w, "alone")


@pytest.mark.parametrize("fmt", FMTS)
def test_values_of_very_different_size_in_a_row(dev, fmt):
    from memory_bound_moe_gb300 import moe_gemv_fp4
    T, N, K = 3, 40, 2048
    x, codes, scales, cd, sd = make(T, N, K, fmt, dev, 8)
    e = torch.randint(-30, 30, (T, K), generator=torch.Generator().manual_seed(1)).float()
    x *= torch.pow(2.0, e).to(dev).to(torch.bfloat16)
    check_gemv(moe_gemv_fp4(x, cd, sd, fmt, 1.0, out_dtype=torch.float32), x, weights64(codes, scales, fmt), "wide")


def test_nonfinite_x_stays_in_its_token(dev):
    from memory_bound_moe_gb300 import moe_gemv_fp4
    x, codes, scales, cd, sd = make(6, 33, 256, "mxfp4", dev, 4)
    codes |= 0x11                                                     # no zero weights
    cd = torch.from_numpy(codes).to(dev)
    clean = moe_gemv_fp4(x, cd, sd, "mxfp4")
    x[1, 100] = float("nan")
    x[4, 3] = float("inf")
    y = moe_gemv_fp4(x, cd, sd, "mxfp4")
    assert y[1].isnan().all() and y[4].isinf().all()
    w = weights64(codes, scales, "mxfp4")[:, 3]
    assert torch.equal(y[4] > 0, torch.from_numpy(w > 0).to(dev))
    for t in (0, 2, 3, 5):
        assert torch.equal(y[t], clean[t])


def test_outputs_behind_the_batch_stay_and_graph_replays(dev):
    from memory_bound_moe_gb300 import moe_gemv_fp4
    T, N, K = 3, 50, 320
    x, codes, scales, cd, sd = make(T, N, K, "nvfp4", dev, 6)
    buf = torch.full((T + 2, N), 7.0, dtype=torch.bfloat16, device=dev)
    moe_gemv_fp4(x, cd, sd, "nvfp4", 2.0, out=buf[:T])
    assert (buf[T:] == 7).all()
    y = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe_gemv_fp4(x, cd, sd, "nvfp4", 2.0, out=y)
    for _ in range(3):
        x.mul_(-2)
        graph.replay()
        assert torch.equal(y, moe_gemv_fp4(x, cd, sd, "nvfp4", 2.0))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    y2 = moe_gemv_fp4(x, cd, sd, "nvfp4", 2.0, stream=s)
    s.synchronize()
    assert torch.equal(y, y2)
    assert moe_gemv_fp4(x[:0], cd, sd, "nvfp4").shape == (0, N)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,N,K", [(2, 17, 1 << 20), (9, 3, (1 << 20) - 32), (32, 70001, 32)])
def test_largest_widths(dev, T, N, K, fmt):
    from memory_bound_moe_gb300 import moe_gemv_fp4
    x, codes, scales, cd, sd = make(T, N, K, fmt, dev, 12)
    y = moe_gemv_fp4(x, cd, sd, fmt, 1.0, out_dtype=torch.float32)
    check_gemv(y, x, weights64(codes, scales, fmt), f"T={T} N={N} K={K}")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [4, 12, 32])
def test_operands_at_16_bytes(dev, fmt, T):
    """Every operand 16, but not 32 bytes behind a boundary: the same bits."""
    from memory_bound_moe_gb300 import moe_gemv_fp4

    def moved(t):
        b = t.contiguous().view(torch.uint8).flatten()
        buf = torch.empty(b.numel() + 64, dtype=torch.uint8, device=dev)
        assert buf.data_ptr() % 32 == 0
        return buf[16:16 + b.numel()].copy_(b).view(t.dtype).view(t.shape)

    for N, K in ((40, 1024), (33, 2880)):
        x, codes, scales, cd, sd = make(T, N, K, fmt, dev, 13)
        y = moe_gemv_fp4(x, cd, sd, fmt, 2.0)
        check_gemv(y, x, weights64(codes, scales, fmt, 2.0 if fmt == "nvfp4" else 1.0), "aligned")
        assert torch.equal(y, moe_gemv_fp4(moved(x), moved(cd), moved(sd), fmt, 2.0))
