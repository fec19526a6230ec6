"""Non-finite weights of an expert reach the tokens that chose it and no
others, whose results keep their bits."""
from __future__ import annotations

import pytest
import torch

from few_reference import BLOCK
from test_gpu_layer import FMTS, Layer, dev, tokens  # noqa: F401

pytestmark = pytest.mark.gpu
NAN_BYTE = {"nvfp4": 127, "mxfp4": 255}


def one_token_on(E, expert, token, T, H, dev, seed):  # noqa: F811
    logits, x = tokens(T, E, H, dev, seed)
    logits[:, expert] = -100.0
    logits[token, expert] = 100.0
    return logits, x


def poisoned(layer, name, expert, row, col, value=float("nan")):
    """The layer with one weight (bfloat16) or one scale byte (4 bits) not
    finite; a function that puts it back."""
    if layer.fmt == "bf16":
        t, at, v = getattr(layer, name), (expert, row, col), value
    else:
        t, at, v = layer.d[1 if name == "w13" else 3], (expert, row, col // BLOCK[layer.fmt]), NAN_BYTE[layer.fmt]
    keep = t[at].clone()
    t[at] = v

    def undo():
        t[at] = keep
    return undo


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [3, 8, 10, 20, 32])
@pytest.mark.parametrize("H,I", [(64, 96), (160, 1120)])
def test_nonfinite_w2_stays_with_its_experts_tokens(dev, T, H, I, fmt):  # noqa: F811
    E, k, e, row = 12, 2, 5, 9
    token = T - 2
    layer = Layer(E, H, I, fmt, dev, 41)
    logits, x = one_token_on(E, e, token, T, H, dev, 42)
    clean = layer(logits, x, k, True)
    assert clean.isfinite().all()
    others = [t for t in range(T) if t != token]
    for value, col in ((float("nan"), 0), (float("inf"), I - 1), (float("-inf"), 40)):
        undo = poisoned(layer, "w2", e, row, col, value)
        out = layer(logits, x, k, True)
        undo()
        assert not out[token, row].isfinite()
        assert torch.equal(out[others], clean[others]), (value, col)
        rest = [h for h in range(H) if h != row]
        assert torch.equal(out[token, rest], clean[token, rest]), (value, col)
    assert torch.equal(layer(logits, x, k, True), clean)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [3, 8, 10, 20])
def test_nonfinite_w13_stays_with_its_experts_tokens(dev, T, fmt):  # noqa: F811
    E, k, e, H, I = 12, 2, 5, 96, 64
    token = T - 1
    layer = Layer(E, H, I, fmt, dev, 43)
    logits, x = one_token_on(E, e, token, T, H, dev, 44)
    clean = layer(logits, x, k, True)
    for row in (3, I + 17):   # gate, up
        undo = poisoned(layer, "w13", e, row, 7)
        out = layer(logits, x, k, True)
        undo()
        assert out[token].isnan().all()
        assert torch.equal(out[:token], clean[:token]), row


@pytest.mark.parametrize("fmt", FMTS)
def test_every_token_of_a_poisoned_expert_and_no_other(dev, fmt):  # noqa: F811
    """Several experts, one of them poisoned and chosen by every third token."""
    T, E, k, H, I = 24, 6, 3, 64, 96
    layer = Layer(E, H, I, fmt, dev, 45)
    logits, x = tokens(T, E, H, dev, 46)
    logits[:, 2] = torch.where(torch.arange(T, device=dev) % 3 == 0, 50.0, -50.0)
    clean = layer(logits, x, k, False)
    undo = poisoned(layer, "w2", 2, 33, 65)
    out = layer(logits, x, k, False)
    undo()
    hit = (torch.arange(T) % 3 == 0).to(dev)
    assert out[hit][:, 33].isnan().all()
    assert torch.equal(out[~hit], clean[~hit])
    rest = [h for h in range(H) if h != 33]
    assert torch.equal(out[:, rest], clean[:, rest])
