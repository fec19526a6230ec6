"""moe_add_rmsnorm and its MXFP8 form on the GPU against the formula in
float64.

Tolerances. residual_out is one float32 addition of two bfloat16 values and
one rounding: exact against the same two operations. out is rounded once to
bfloat16 (half a step, at most 2^-8 of the value); before that float32: the
sum of squares (a tree of at most 15 levels plus at most 32 sequential adds
per thread: under 64 roundings of 2^-24, halved by the square root), rsqrt (2
ulp) and four products: under 64 * 2^-24 = 2^-18 relative in all. So
|got - ref| <= (2^-8 + 2^-17) |ref| + 2^-133 (the subnormal step). MXFP8 codes
and scales are the oracle's quantization of the very bfloat16 rows: exact."""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

RTOL = 2.0 ** -8 + 2.0 ** -17
ATOL = 2.0 ** -133


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from memory_bound_moe_gb300 import build
    build.build()
    return torch.device("cuda:0")


def offset16(t):
    """A copy that starts 16 but not 32 bytes off a 32-byte boundary."""
    buf = torch.empty(t.numel() + 16, dtype=t.dtype, device=t.device)
    shift = ((16 - buf.data_ptr() % 32) % 32) // t.element_size()
    v = buf[shift:shift + t.numel()].view(t.shape)
    v.copy_(t)
    assert v.data_ptr() % 32 == 16
    return v


def inputs(T, H, dev, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    row = torch.exp(spread * torch.randn(T, 1, generator=g))
    x = (torch.randn(T, H, generator=g) * row).to(torch.bfloat16)
    r = (torch.randn(T, H, generator=g) * row * 2).to(torch.bfloat16)
    w = (1 + 0.2 * torch.randn(H, generator=g)).to(torch.bfloat16)
    return x.to(dev), r.to(dev), w.to(dev)


def reference(x, r, w, bias, eps):
    h = x.double().cpu() + (r.double().cpu() if r is not None else 0)
    y = (w.double().cpu() + bias) * h / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    return h, y


def check_out(got, ref, what):
    err = (got.double().cpu() - ref).abs()
    bad = err > RTOL * ref.abs() + ATOL
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist())


SHAPES = [(1, 8), (3, 16), (1, 256), (16, 7168), (33, 264), (257, 2880), (1023, 2880), (4096, 2048), (100, 520),
          (2, 16384), (3, 16392), (2, 32776), (2, 65536), (2, 65552)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("wide", [True, False])
def test_add_rmsnorm(dev, T, H, wide):
    from memory_bound_moe_gb300 import moe_add_rmsnorm
    x, r, w = inputs(T, H, dev, T * 31 + H)
    if not wide:
        x = offset16(x)
    keep = r.clone()
    y, ro = moe_add_rmsnorm(x, r, w, 0.0, 1e-6, residual_out=torch.full_like(r, float("nan")))
    assert torch.equal(r, keep)                                       # apart: the input stays
    h, ref = reference(x, r, w, 0.0, 1e-6)
    check_out(y, ref, f"T={T} H={H}")
    assert torch.equal(ro, (x.float() + r.float()).to(torch.bfloat16))
    # in place gives the same bits, and so does a second run
    y2, ro2 = moe_add_rmsnorm(x, r, w, 0.0, 1e-6)
    assert ro2.data_ptr() == r.data_ptr()
    assert torch.equal(y2, y) and torch.equal(r, ro)


@pytest.mark.parametrize("T,H", [(1, 64), (50, 2880), (9, 20480)])
@pytest.mark.parametrize("bias", [0.0, 1.0])
def test_without_residual_and_with_bias(dev, T, H, bias):
    from memory_bound_moe_gb300 import moe_add_rmsnorm
    x, _, w = inputs(T, H, dev, H)
    y, ro = moe_add_rmsnorm(x, None, w, bias, 1e-5)
    assert ro is None
    check_out(y, reference(x, None, w, bias, 1e-5)[1], "no residual")


@pytest.mark.parametrize("T,H", [(1, 32), (7, 96), (16, 7168), (1023, 2880), (4096, 2048), (3, 16416), (2, 65568)])
@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("both", [True, False])
def test_mxfp8_quantizes_the_bf16_rows(dev, oracle_mod, T, H, wide, both):
    from memory_bound_moe_gb300 import moe_add_rmsnorm, moe_add_rmsnorm_mxfp8
    x, r, w = inputs(T, H, dev, T + H)
    w[:32] = 0                                                        # an all-zero block
    if not wide:
        x = offset16(x)
    y, ro = moe_add_rmsnorm(x, r, w, residual_out=torch.empty_like(r))
    out = torch.empty_like(y) if both else None
    codes, scales, ro2 = moe_add_rmsnorm_mxfp8(x, r, w, out=out, residual_out=torch.empty_like(r))
    if both:
        assert torch.equal(out, y)
    assert torch.equal(ro, ro2)
    c, s = oracle_mod.quant_mxfp8(y.cpu().view(torch.int16).numpy().view(np.uint16))
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), c)


def test_special_rows(dev):
    """A zero row, a cancelling row, NaN and infinity kept in their own rows."""
    from memory_bound_moe_gb300 import moe_add_rmsnorm
    H = 512
    x, r, w = inputs(6, H, dev, 5, 0.0)
    x[0] = 0
    r[0] = 0
    r[1] = -x[1]
    x[2, 7] = float("nan")
    x[3, 9] = float("inf")
    y, ro = moe_add_rmsnorm(x, r, w, 0.0, 1e-6, residual_out=torch.empty_like(r))
    assert (y[0] == 0).all() and (y[1] == 0).all()
    assert y[2].isnan().all()
    assert y[3, 9].isnan() and ro[3, 9] == float("inf")
    check_out(y[4:], reference(x[4:], r[4:], w, 0.0, 1e-6)[1], "rows beside them")


def test_rows_behind_the_batch_stay(dev):
    from memory_bound_moe_gb300 import moe_add_rmsnorm_mxfp8
    T, H = 5, 96
    x, r, w = inputs(T, H, dev, 9)
    big = lambda shape, dt, v: torch.full(shape, v, dtype=dt, device=dev)
    y, ro = big((T + 3, H), torch.bfloat16, 7.0), big((T + 3, H), torch.bfloat16, 7.0)
    c, s = big((T + 3, H), torch.uint8, 171), big((T + 3, H // 32), torch.uint8, 205)
    moe_add_rmsnorm_mxfp8(x, r, w, codes=c[:T], scales=s[:T], out=y[:T], residual_out=ro[:T])
    assert (y[T:] == 7).all() and (ro[T:] == 7).all() and (c[T:] == 171).all() and (s[T:] == 205).all()


def test_side_stream_and_graph(dev):
    from memory_bound_moe_gb300 import moe_add_rmsnorm
    x, r, w = inputs(64, 2048, dev, 3)
    y, ro = moe_add_rmsnorm(x, r, w, residual_out=torch.empty_like(r))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y2, ro2 = moe_add_rmsnorm(x, r, w, residual_out=torch.empty_like(r), stream=s)
    s.synchronize()
    assert torch.equal(y, y2) and torch.equal(ro, ro2)
    y3, ro3 = torch.empty_like(y), torch.empty_like(r)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe_add_rmsnorm(x, r, w, out=y3, residual_out=ro3)
    for k in range(3):
        x.mul_(2 if k else 1)
        y3.zero_()
        g.replay()
        want = moe_add_rmsnorm(x, r, w, residual_out=torch.empty_like(r))
        assert torch.equal(y3, want[0]) and torch.equal(ro3, want[1])


def test_empty_batch(dev):
    from memory_bound_moe_gb300 import moe_add_rmsnorm, moe_add_rmsnorm_mxfp8
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=dev)
    w = torch.ones(64, dtype=torch.bfloat16, device=dev)
    y, _ = moe_add_rmsnorm(x, x.clone(), w)
    assert y.shape == (0, 64)
    codes, scales, _ = moe_add_rmsnorm_mxfp8(x, None, w)
    assert codes.shape == (0, 64) and scales.shape == (0, 2)
