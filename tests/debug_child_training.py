"""Child process of test_debug_build_training: runs with MOE_LIB_PATH naming the bounds-checked
library (built with -DMOE_DEBUG).

Clean inputs raise no flag; then one out-of-range index each (a row segment, a sorted_idx
value), which the checked kernels keep from being used and flag (an inv_idx out of range is a
dropped assignment, in every build).  The planted cases run only after moe_debug_take has
succeeded, i.e. only on the checked build.  Prints one line per step and "DEBUG CHILD OK" at the
end.
"""
from __future__ import annotations

import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))

import torch  # noqa: E402

import moe_expert_ffn_router_amd as moe  # noqa: E402

DEV = torch.device("cuda")
BF = torch.bfloat16


def expect(flag: int, what: str) -> None:
    torch.cuda.synchronize()
    got = moe.moe_debug_take()
    print(f"{what}: flags {got:#x}", flush=True)
    assert got == flag, (what, got, flag)


def ffn(per: int) -> None:
    E, H, I, k = 4, 256, 128, 2
    A = E * per
    rec = (torch.randn(E, 3 * H * I, device=DEV) * 0.05).to(BF)
    W = moe.experts("bf16", E, H, I, rec, rec.shape[1] * 2)
    x = torch.randn(A // k, H, device=DEV).to(BF)
    gu, y = torch.zeros(A, 2 * I, dtype=BF, device=DEV), torch.zeros(A, H, dtype=BF, device=DEV)
    dx, d13, d2 = torch.zeros_like(y), torch.zeros(E, 2 * I, H, device=DEV), torch.zeros(E, H, I, device=DEV)
    ws = torch.empty(moe.moe_expert_ffn_backward_workspace(W, A // k, k), dtype=torch.uint8, device=DEV)
    for what, flag in (("clean", 0), ("segment", moe.DBG_SEGMENT), ("start", moe.DBG_SEGMENT),
                       ("sorted", moe.DBG_SORTED), ("negative", moe.DBG_SORTED)):
        counts = torch.full((E,), per, dtype=torch.int32, device=DEV)
        off = (torch.arange(E + 1, device=DEV) * per).int()
        order = torch.randperm(A, device=DEV).int()
        if what == "segment":
            off[E - 1] = A - 1
        if what == "start":
            off[1] = -3
        if what == "sorted":
            order[5] = A + 40
        if what == "negative":
            order[A - 1] = -7
        moe.moe_expert_ffn_train(W, x, A // k, k, counts, off, order, gu, y, ws)
        expect(flag, f"train per={per} {what}")
        moe.moe_expert_ffn_backward(W, x, A // k, k, counts, off, order, gu, y, ws, dx, d13, d2)
        expect(flag, f"backward per={per} {what}")


if __name__ == "__main__":
    moe.moe_debug_take()  # raises on a release build
    for per in (2, 40, 100, 300):
        ffn(per)
    print("DEBUG CHILD OK", flush=True)
