"""The expert training calls where segments leave gaps: places of fixed length for each expert, some of
them empty, with rows behind the last.  Entries of sorted_idx that no expert owns may hold anything (here:
-1, 2^31 - 1, numbers of tokens that do not exist), and the rows of gate_up and d_y_perm there NaN.
What comes out is, bit by bit, what a valid permutation and ordinary values there give.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_cases import flush
from train_tiles import sides

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from test_gpu_expert_train import BF, DEV, F32, Case, check_backward, check_forward  # noqa: E402

# places of `place` rows (the last may be full), experts without rows first, last and between; the tiles that
# the gathered gradient of w13, gate/up and dh take
CASES = [
    (dict(counts=[0, 3, 0, 40, 0], place=40, H=256, I=128, k=1), (64, 64, 64)),
    (dict(counts=[0, 100, 0, 0, 64, 1, 0, 99, 0], place=100, H=1024, I=256, k=3), (128, 64, 64)),
    (dict(counts=[0, 180, 0, 0, 70, 64, 1, 300, 0, 129, 320, 33, 0], place=320, H=1024, I=640, k=1), (256, 128, 64)),
    (dict(counts=[0, 180, 0, 0, 70, 64, 1, 300, 0, 129, 320, 33, 0], place=320, H=1024, I=640, k=3), (256, 128, 64)),
    (dict(counts=[0, 600, 0, 257, 64, 0, 511, 0], place=600, H=2048, I=1024, k=2), (256, 256, 128)),
    (dict(counts=[0] * 90 + [17] + [0] * 210, place=20, H=256, I=256, k=3), (256, 128, 128)),
]


def gaps(c, place, k):
    """Moves the case's rows to places of `place` rows each, with a gap before the first and behind the last."""
    E, first = c.E, 7
    A = -(-(first + E * place + 5) // k) * k
    at = first + np.concatenate([np.arange(n) + e * place for e, n in enumerate(np.diff(c.ends))]).astype(int)
    at = torch.from_numpy(at).to(DEV)
    g = torch.Generator(device=DEV).manual_seed(5)
    tokens = A // k
    c.x = torch.randn(tokens, c.H, generator=g, device=DEV).to(BF)
    order = torch.randperm(A, generator=g, device=DEV).int()
    owned = order[at]
    c.rows = c.x[owned.long() // k]
    gu, dy = c.gu[:c.n].clone(), c.dy[:c.n].clone()
    c.gu = torch.randn(A, 2 * c.I, generator=g, device=DEV).to(BF)
    c.dy = torch.randn(A, c.H, generator=g, device=DEV).to(BF)
    c.gu[at], c.dy[at] = gu, dy
    c.T, c.k, c.A, c.sorted_idx = tokens, k, A, order
    c.offsets = torch.tensor([first + e * place for e in range(E)] + [A], dtype=torch.int32, device=DEV)
    import moe_expert_ffn_router_amd as moe
    c.ws = torch.full((moe.moe_expert_ffn_backward_workspace(c.W, tokens, k),), 255, dtype=torch.uint8, device=DEV)
    return at


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("spec,tiles", CASES, ids=[f"{len(s['counts'])}e{s['H']}x{s['I']}k{s['k']}" for s, _ in CASES])
def test_entries_that_no_expert_owns(spec, tiles, dtype):
    flush(f"[train] gaps {len(spec['counts'])} experts H={spec['H']} I={spec['I']} k={spec['k']} {dtype}")
    c = Case(spec["counts"], spec["H"], spec["I"], seed=30)
    at = gaps(c, spec["place"], spec["k"])
    s = sides(c.E, c.H, c.I, c.A)
    assert (s["w13"], s["gate_up"], s["dh"]) == tiles
    want = (*c.forward(), *c.backward(dtype))
    free = torch.ones(c.A, dtype=torch.bool, device=DEV)
    free[at] = False
    junk = torch.tensor([-1, 2 ** 31 - 1, c.A, -2 ** 31, c.A + 12345, -7], dtype=torch.int32, device=DEV)
    c.sorted_idx[free] = junk.repeat(c.A)[:int(free.sum())]
    c.gu[free], c.dy[free] = float("nan"), float("nan")
    got = (*c.forward(), *c.backward(dtype))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a.nan_to_num(nan=7.0), b.nan_to_num(nan=7.0)) and not bool(b.isnan().any())
    # and by the formulas: the rows in the order of the experts
    gu, y, dx, d13, d2 = got
    for t in (gu, y, dx):
        assert bool((t[free] == 3.5).all())
    kept = c.gu, c.dy
    c.gu, c.dy = c.gu[at], c.dy[at]
    check_forward(c, gu[at], y[at])
    check_backward(c, dx[at], d13, d2)
    c.gu, c.dy = kept
