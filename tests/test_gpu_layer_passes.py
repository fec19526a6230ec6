"""moe_layer_fp4 where one expert has more than 16 tokens (two passes over its
weights) and the widths take several slices of k: against float64 (bounds:
few_reference.py)."""
from __future__ import annotations

import pytest
import torch

from test_gpu_layer import Layer, dev, run_and_check, tokens  # noqa: F401

pytestmark = pytest.mark.gpu
FMTS = ["nvfp4", "mxfp4"]
TOKENS = [17, 20, 24, 25, 32]   # 16 + 1, 4, 8: a second pass of one group; 16 + 9, 16: of two


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("I", [5664, 8192, 14336])
@pytest.mark.parametrize("T", TOKENS)
def test_second_pass_over_several_slices_of_fc2(dev, T, I, fmt):  # noqa: F811
    """Every expert with every token: a block's share of an expert is longer
    than one slice of 11 chunks for two groups of tokens."""
    H = 32
    layer = Layer(8, H, I, fmt, dev, I)
    logits, x = tokens(T, 8, H, dev, T)
    run_and_check(layer, logits, x, 8, True, f"T={T} I={I} {fmt}, k = E")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [17, 23, 32])
def test_one_expert_above_16_among_others(dev, T, fmt):  # noqa: F811
    """Experts with 0, a few and more than 16 tokens in one batch, the shares
    of fc2's blocks beginning and ending inside them."""
    E, H, I = 9, 64, 14336
    layer = Layer(E, H, I, fmt, dev, 5)
    logits, x = tokens(T, E, H, dev, 50 + T)
    logits[:, 4] = 30.0                      # every token
    logits[: T // 2 + 9, 7] = 20.0           # 17 and more
    logits[:, 0] = -50.0                     # none
    run_and_check(layer, logits, x, 5, True, f"T={T} skewed {fmt}")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("I", [5664, 14336])
@pytest.mark.parametrize("T", TOKENS)
def test_all_tokens_on_one_expert(dev, T, I, fmt):  # noqa: F811
    H = 64
    layer = Layer(3, H, I, fmt, dev, I + 1)
    logits, x = tokens(T, 3, H, dev, T + 1)
    logits[:, 1] = 40.0
    run_and_check(layer, logits, x, 1, True, f"T={T} I={I} {fmt}, one expert")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("H", [5664, 14336])
@pytest.mark.parametrize("T", TOKENS)
def test_second_pass_over_several_fillings_of_fc1(dev, T, H, fmt):  # noqa: F811
    I = 64
    layer = Layer(3, H, I, fmt, dev, H)
    logits, x = tokens(T, 3, H, dev, T + 2)
    run_and_check(layer, logits, x, 3, True, f"T={T} H={H} {fmt}, k = E")
    logits[:, 1] = 40.0
    run_and_check(layer, logits, x, 1, True, f"T={T} H={H} {fmt}, one expert")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,H,I", [(8, 11296, 96), (5, 64, 11808), (16, 64, 12320), (10, 6176, 6176)])
def test_several_slices_of_one_pass(dev, T, H, I, fmt):  # noqa: F811
    layer = Layer(2, H, I, fmt, dev, 3)
    logits, x = tokens(T, 2, H, dev, T + 3)
    run_and_check(layer, logits, x, 2, False, f"T={T} H={H} I={I} {fmt}")
