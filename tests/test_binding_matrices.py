"""What the bindings take for a matrix (no GPU needed: the refusals come before any device is asked)."""
from __future__ import annotations

from types import SimpleNamespace

import numpy as np
import pytest
import torch

import moe_expert_ffn_router_amd as moe


@pytest.mark.parametrize("bad", [np.zeros((4, 8), np.float32), SimpleNamespace(shape=(4, 8)), [[1.0]], None,
                                 torch.zeros(4), torch.zeros(4, 8, 1), torch.zeros(())],
                         ids=["array", "shape", "list", "none", "1d", "3d", "0d"])
def test_only_matrices_of_torch(bad):
    """One exception type for all of them, whichever call is given them."""
    with pytest.raises(ValueError, match="expected a matrix"):
        moe.moe_route_backward(bad, 1, None, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="expected a matrix"):
        moe.moe_fp8_quantize(bad, None, None)
    with pytest.raises(ValueError, match="expected a matrix"):
        moe.moe_dispatch(bad, None, 1, torch.zeros(4, 8))
    with pytest.raises(ValueError, match="expected a matrix"):
        moe.moe_dispatch(torch.zeros(4, 8), None, 1, bad)


@pytest.mark.parametrize("rows", [2 ** 31, 2 ** 32, 2 ** 32 + 4])
def test_sizes_past_32_bits(rows):
    """The library takes 32-bit sizes: 2^32 rows are not cut to none (all of whose assignments would be
    dropped in silence)."""
    big, x = torch.empty((rows, 8), dtype=torch.bfloat16, device="meta"), torch.zeros(4, 8)
    for call in (lambda: moe.moe_dispatch(x, None, 1, big), lambda: moe.moe_dispatch(big, None, 1, x),
                 lambda: moe.moe_dispatch_backward(big, None, 1, x),
                 lambda: moe.moe_combine_backward(x, None, None, 1, big),
                 lambda: moe.moe_fp8_quantize(torch.empty((8, rows), device="meta"), None, None)):
        with pytest.raises(ValueError, match=f"{rows}.*32 bits"):
            call()
