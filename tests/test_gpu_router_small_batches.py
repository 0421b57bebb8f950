"""moe_balance_loss on one chunk of rows in a few and in many sequences: both sides of the rule
that lets one kernel finish the loss, against the float64 oracle (test_gpu_router_training's
tolerances)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_cases import flush

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from test_gpu_router_training import Batch  # noqa: E402


@pytest.mark.parametrize("T,E,k", [(64, 256, 8), (128, 60, 4), (128, 1024, 16), (31, 17, 3), (0, 8, 2)])
@pytest.mark.parametrize("S", [1, 3, 4, 5, 6, 64, 256, 257])
def test_one_chunk(T, E, k, S):
    flush(f"[router, one chunk] T={T} E={E} k={k} S={S}")
    rng = np.random.default_rng(T + S)
    seq = np.sort(rng.integers(0, T + 1, S + 1)).astype(np.int32)
    if S == 64 and T == 64:
        seq = np.arange(65, dtype=np.int32)              # one row each
    Batch(T, E, k, list(seq), masked=S % 2 == 0, seed=T + S).run()
