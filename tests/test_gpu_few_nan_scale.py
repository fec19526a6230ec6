"""A scale byte that encodes NaN makes its own row of the product NaN; all
other rows keep their bits, also those that share a tile of 16 with it and end
inside a chunk of k."""
from __future__ import annotations

import pytest
import torch

from few_reference import BLOCK
from test_gpu_gemv_fp4 import make
from test_gpu_layer import dev  # noqa: F401

pytestmark = pytest.mark.gpu
NAN_BYTE = {"nvfp4": 127, "mxfp4": 255}


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("K", [32, 768, 1024, 2880])
@pytest.mark.parametrize("T", [1, 9, 20])
def test_a_nan_scale_makes_its_row_nan_and_no_other(dev, T, K, fmt):  # noqa: F811
    from memory_bound_moe_gb300 import moe_gemv_fp4
    N = 40
    x, codes, scales, cd, sd = make(T, N, K, fmt, dev, 31)
    clean = moe_gemv_fp4(x, cd, sd, fmt, out_dtype=torch.float32)
    assert clean.isfinite().all()
    for row, block in ((5, K // BLOCK[fmt] - 1), (38, 0)):
        bad = scales.copy()
        bad[row, block] = NAN_BYTE[fmt]
        y = moe_gemv_fp4(x, cd, torch.from_numpy(bad).to(dev), fmt, out_dtype=torch.float32)
        assert y[:, row].isnan().all()
        rest = [n for n in range(N) if n != row]
        assert torch.equal(y[:, rest], clean[:, rest]), (row, block)
