"""Calls that feed each other with nothing but this library's launches between
them: every launch may start before the one in front of it has ended, and must
not read early."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from few_reference import random_fp4
from test_gpu_layer import FMTS, Layer, dev, tokens  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [2, 12])
def test_chained_calls_with_one_workspace(dev, T, fmt):  # noqa: F811
    """norm -> router product -> layer -> layer -> norm ..., over buffers that
    are used again at once: the same bits as with a wait after every call."""
    from memory_bound_moe_gb300 import moe_add_rmsnorm, moe_gemv_fp4, moe_layer_workspace_size
    E, k, H, I = 16, 4, 256, 160
    layer = Layer(E, H, I, fmt, dev, 61)
    rc, rs = (torch.from_numpy(a).to(dev) for a in random_fp4(np.random.default_rng(62), (E, H), "nvfp4"))
    weight = torch.ones(H, dtype=torch.bfloat16, device=dev)
    _, x0 = tokens(T, E, H, dev, 63)
    ws = torch.empty(moe_layer_workspace_size(T, E, k, H, I), dtype=torch.uint8, device=dev)
    y, h, h2 = (torch.empty_like(x0) for _ in range(3))
    logits = torch.empty((T, E), dtype=torch.float32, device=dev)

    def chain(wait):
        seen = []
        h.copy_(x0)
        torch.cuda.synchronize()
        for _ in range(40):
            for call in (lambda: moe_add_rmsnorm(h, None, weight, out=y),
                         lambda: moe_gemv_fp4(y, rc, rs, "nvfp4", 300.0, out=logits),
                         lambda: layer(logits, y, k, True, out=h2, workspace=ws),
                         lambda: layer(logits, h2, k, True, out=h, workspace=ws)):
                call()
                if wait:
                    torch.cuda.synchronize()
            if wait:
                seen.append(h.clone())
        torch.cuda.synchronize()
        return seen, h.clone(), logits.clone()

    seen, want, want_logits = chain(True)
    assert want.isfinite().all() and (want != 0).any()
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[-2], seen[-1])   # every step counts
    for _ in range(5):
        _, got, got_logits = chain(False)
        assert torch.equal(got, want) and torch.equal(got_logits, want_logits)
