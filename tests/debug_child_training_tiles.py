"""Child process of test_debug_build_training_tiles: runs with MOE_LIB_PATH naming the bounds-checked
library (built with -DMOE_DEBUG).

Expert training calls in tiles of 256 x 256 and 128 x 128.  Clean inputs raise no flag, among them segments with
gaps whose index entries belong to no expert and hold anything; then one out-of-range index each (a row
segment, a sorted_idx value), which the checked kernels keep from being used and flag.  The planted cases run
only after moe_debug_take has succeeded, i.e. only on the checked build.  Prints one line per step and "DEBUG
CHILD OK" at the end.
"""
from __future__ import annotations

import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, HERE)
sys.path.insert(0, os.path.dirname(HERE))

import torch  # noqa: E402

import moe_expert_ffn_router_amd as moe  # noqa: E402
from train_tiles import sides  # noqa: E402

DEV = torch.device("cuda")
BF = torch.bfloat16
# E, rows of an expert, H, I
SIZES = [(8, 600, 2048, 1024), (4, 1100, 1024, 2048), (5, 1000, 1024, 512), (6, 400, 2048, 1024)]


def expect(flag: int, what: str) -> None:
    torch.cuda.synchronize()
    got = moe.moe_debug_take()
    print(f"{what}: flags {got:#x}", flush=True)
    assert got == flag, (what, got, flag)


def ffn(E: int, per: int, H: int, I: int, gathered: bool) -> None:
    k = 2 if gathered else 1
    A = E * per
    rec = (torch.randn(E, 3 * H * I, device=DEV) * 0.05).to(BF)
    W = moe.experts("bf16", E, H, I, rec, rec.shape[1] * 2)
    x = torch.randn(A // k, H, device=DEV).to(BF)
    gu, y = torch.zeros(A, 2 * I, dtype=BF, device=DEV), torch.zeros(A, H, dtype=BF, device=DEV)
    dx, d13, d2 = torch.zeros_like(y), torch.zeros(E, 2 * I, H, device=DEV), torch.zeros(E, H, I, device=DEV)
    ws = torch.empty(moe.moe_expert_ffn_backward_workspace(W, A // k, k), dtype=torch.uint8, device=DEV)
    cases = [("clean", 0), ("gaps", 0), ("segment", moe.DBG_SEGMENT), ("start", moe.DBG_SEGMENT)]
    if gathered:
        cases += [("sorted", moe.DBG_SORTED), ("negative", moe.DBG_SORTED)]
    for what, flag in cases:
        counts = torch.full((E,), per, dtype=torch.int32, device=DEV)
        off = (torch.arange(E + 1, device=DEV) * per).int()
        order = torch.randperm(A, device=DEV).int()
        if what == "gaps":  # the first and the last but one without rows, the others short
            counts -= torch.arange(E, device=DEV).int() * 7 + 1
            counts[0] = counts[E - 2] = 0
            free = torch.arange(A, device=DEV) % per >= counts.repeat_interleave(per)
            order[free] = torch.tensor([-1, 2 ** 31 - 1], dtype=torch.int32, device=DEV).repeat(A)[:int(free.sum())]
        if what == "segment":
            off[E - 1] = A - 1
        if what == "start":
            off[1] = -3
        if what == "sorted":
            order[5] = A + 40
        if what == "negative":
            order[A - 1] = -7
        idx = order if gathered else None
        name = f"{E} x {per} of {H} x {I}, {'gathered' if gathered else 'in order'}, {what}"
        moe.moe_expert_ffn_train(W, x, A // k, k, counts, off, idx, gu, y, ws)
        expect(flag, f"train {name}")
        moe.moe_expert_ffn_backward(W, x, A // k, k, counts, off, idx, gu, y, ws, dx, d13, d2)
        expect(flag, f"backward {name}")


if __name__ == "__main__":
    taken = {(n, s) for E, per, H, I in SIZES for n, s in sides(E, H, I, E * per).items()}
    missing = {(n, s) for n in ("gate_up", "down", "dh", "dx", "w13", "w2") for s in (128, 256)} - taken
    assert not missing, missing
    moe.moe_debug_take()  # raises on a release build
    for size in SIZES:
        for gathered in (True, False):
            ffn(*size, gathered)
    print("DEBUG CHILD OK", flush=True)
