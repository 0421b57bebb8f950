"""moe_dispatch, moe_dispatch_backward and moe_combine_backward over more tokens than one grid of fewer than
2^32 threads holds (a token a workgroup of 256 above 512 columns, four below), up to the 2^27 assignments that
they take.  The values are whole numbers whose sums are exact, so results are compared bit by bit.
"""
from __future__ import annotations

import pytest
import torch

from gpu_cases import flush

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_expert_ffn_router_amd as moe  # noqa: E402

DEV = torch.device("cuda")
BF = torch.bfloat16
STEP = 1 << 20


def numbers(first, n, H, salt):
    """Rows first .. first + n of whole numbers 0 to 15 that differ from row to row."""
    r = torch.arange(first, first + n, device=DEV, dtype=torch.int32)[:, None] * -1640531535 + salt
    c = torch.arange(H, device=DEV, dtype=torch.int32)[None] * 40503
    return (((r + c) >> 9) & 15).to(BF)


def table(n, H, salt):
    t = torch.empty(n, H, dtype=BF, device=DEV)
    for at in range(0, n, STEP):
        t[at:at + STEP] = numbers(at, min(STEP, n - at), H, salt)
    return t


@pytest.mark.parametrize("T,k,H", [((1 << 24) + 3, 1, 520), ((1 << 26) + 7, 1, 8), (1 << 26, 2, 8),
                                   ((1 << 25) + 1, 1, 16)])
def test_more_tokens_than_a_grid_holds(T, k, H):
    flush(f"[rows] many T={T} k={k} H={H}")
    A = T * k
    x = table(T, H, 1)
    inv = torch.arange(A - 1, -1, -1, dtype=torch.int32, device=DEV)      # row A - 1 - a
    slice_ = (1 << 23) * (1 if H > 512 else 4)
    lost = sorted({0, A - 1, min(slice_, T - 1) * k, min(2 * slice_, T - 1) * k - 1})
    inv[lost] = -1
    rows = torch.full((A, H), 3.5, dtype=BF, device=DEV)
    moe.moe_dispatch(x, inv, k, rows)
    torch.cuda.synchronize()
    for at in range(0, T, STEP):
        n = min(STEP, T - at)
        want = x[at:at + n].repeat_interleave(k, 0)
        for a in lost:
            if at * k <= a < (at + n) * k:
                want[a - at * k] = 3.5
        assert torch.equal(rows[A - (at + n) * k:A - at * k].flip(0), want), at
    # sums, with an addend, weights of one half and the dots
    w = torch.full((T, k), 0.5, device=DEV)
    dx, dw = torch.full((T, H), 3.5, dtype=BF, device=DEV), torch.full((T, k), 3.5, device=DEV)
    moe.moe_dispatch_backward(rows, inv, k, dx, topk_w=w, d_add=x, x=x, d_topk_w=dw)
    dw2 = torch.full((T, k), 3.5, device=DEV)
    out = torch.full((A, H), 3.5, dtype=BF, device=DEV)
    moe.moe_combine_backward(x, inv, w, k, out, y_perm=rows, d_topk_w=dw2)
    torch.cuda.synchronize()
    for at in range(0, T, STEP):
        n = min(STEP, T - at)
        p = x[at:at + n].float()
        there = torch.ones(n * k, device=DEV)
        for a in lost:
            if at * k <= a < (at + n) * k:
                there[a - at * k] = 0.0
        there = there.view(n, k)
        assert torch.equal(dx[at:at + n], (p + 0.5 * there.sum(1, keepdim=True) * p).to(BF)), at
        dots = (p * p).sum(1, keepdim=True) * there
        assert torch.equal(dw[at:at + n], dots) and torch.equal(dw2[at:at + n], dots), at
        half = (0.5 * p).to(BF).repeat_interleave(k, 0)
        half[there.view(-1) == 0] = 3.5
        assert torch.equal(out[A - (at + n) * k:A - at * k].flip(0), half), at
