"""Child process of test_debug_build_router_fp8: runs with MOE_LIB_PATH naming the
bounds-checked library (built with -DMOE_DEBUG).

Clean inputs raise no flag; then one out-of-range index each (sequence offsets, an expert's
row segment, a slot, a sorted_idx value), which the checked kernels replace by an in-range one
and flag.  The planted cases run only after moe_debug_take has succeeded, i.e. only on the
checked build.  Prints one line per step and "DEBUG CHILD OK" at the end.
"""
from __future__ import annotations

import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))

import torch  # noqa: E402

import moe_expert_ffn_router_amd as moe  # noqa: E402

DEV = torch.device("cuda")


def expect(flag: int, what: str) -> None:
    torch.cuda.synchronize()
    got = moe.moe_debug_take()
    print(f"{what}: flags {got:#x}", flush=True)
    assert got == flag, (what, got, flag)


def router(T: int, E: int) -> None:
    g = torch.Generator(device=DEV).manual_seed(T)
    lg = torch.randn(T, E, device=DEV, generator=g)
    ids = torch.topk(lg, 2, 1).indices.int().contiguous()
    w = torch.rand(T, 2, device=DEV, generator=g)
    n, c = torch.zeros(3, dtype=torch.int32, device=DEV), torch.zeros(3, E, dtype=torch.int32, device=DEV)
    p, l, dl = torch.zeros(3, E, device=DEV), torch.zeros(3, device=DEV), torch.ones(3, device=DEV)
    out = torch.zeros(T, E, device=DEV)
    ws = torch.empty(moe.moe_balance_loss_workspace(T, E, 3), dtype=torch.uint8, device=DEV)
    for seq, flag in (([0, T // 3, T // 2, T], 0), ([0, T // 3, T // 2, T + 77], moe.DBG_SEGMENT),
                      ([-5, T // 3, T // 2, T], moe.DBG_SEGMENT),
                      ([0, T // 2, T // 3, T], moe.DBG_SEGMENT)):
        s = torch.tensor(seq, dtype=torch.int32, device=DEV)
        moe.moe_balance_loss(lg, ids, 2, n, c, p, l, ws, seq_offsets=s)
        expect(flag, f"balance T={T} E={E} seq={seq}")
        moe.moe_route_backward(lg, 2, ids, w, w, n, c, dl, out, seq_offsets=s)
        expect(flag, f"gradient T={T} E={E} seq={seq}")


def product(E: int, per: int, N: int, K: int) -> None:
    M = E * per
    code = lambda *s: torch.randint(0, 0x70, s, dtype=torch.uint8, device=DEV)  # noqa: E731
    a, w = code(M, K), code(E, N, K)
    sa = torch.rand(M, -(-K // 128), device=DEV)
    sw = torch.rand(E, -(-N // 128), -(-K // 128), device=DEV)
    y = torch.zeros(M, N, dtype=torch.bfloat16, device=DEV)
    counts = torch.full((E,), per, dtype=torch.int32, device=DEV)
    off = (torch.arange(E + 1, device=DEV) * per).int()
    moe.moe_fp8_matmul(a, sa, w, sw, y, None, counts, off)
    expect(0, f"product E={E} rows={per} N={N} K={K}")
    counts[-1] += 40
    moe.moe_fp8_matmul(a, sa, w, sw, y, None, counts, off)
    expect(moe.DBG_SEGMENT, f"product E={E} rows={per}: segment past the rows")
    counts[-1] -= 40
    off[0] = -3
    moe.moe_fp8_matmul(a, sa, w, sw, y, None, counts, off)
    expect(moe.DBG_SEGMENT, f"product E={E} rows={per}: segment before the rows")


def ffn(E: int, T: int, k: int, H: int, I: int) -> None:
    L = moe.moe_expert_layout_query("fp8_b128", H, I)
    base = torch.randint(0, 0x70, (E, L["stride"]), dtype=torch.uint8, device=DEV)
    for o, n in ((L["w13_scale"], 2 * I * H // 16384), (L["w2_scale"], I * H // 16384)):
        base[:, o:o + n * 4] = (torch.rand(E, n, device=DEV) * 1e-4).view(torch.uint8)
    W = moe.experts("fp8_b128", E, H, I, base, L["stride"])
    A = T * k
    per = A // E
    counts = torch.full((E,), per, dtype=torch.int32, device=DEV)
    off = (torch.arange(E + 1, device=DEV) * per).int()
    srt = torch.randperm(A, device=DEV).int()
    slots = torch.randperm(E, device=DEV).int()
    x = torch.randn(T, H, device=DEV).bfloat16()
    y = torch.zeros(A, H, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(moe.moe_expert_ffn_fp8_workspace(W, T, k), dtype=torch.uint8, device=DEV)

    def call():
        moe.moe_expert_ffn_fp8(W, slots, x, T, k, counts, off, srt, y, ws)

    call()
    expect(0, f"ffn E={E} T={T} k={k}")
    keep = int(slots[1])
    slots[1] = E + 5
    call()
    expect(moe.DBG_SLOT, f"ffn E={E} T={T}: slot")
    slots[1] = keep
    keep = int(srt[3])
    srt[3] = A + 1000
    call()
    expect(moe.DBG_SORTED, f"ffn E={E} T={T}: sorted index")
    srt[3] = keep


def main() -> None:
    torch.cuda.synchronize()
    assert moe.moe_debug_take() == 0   # raises on a release build
    router(100, 16)
    router(2000, 300)
    product(4, 3, 96, 272)             # 16-row tiles
    product(4, 40, 96, 272)            # 64 x 64
    product(40, 50, 1100, 272)         # 64 x 256
    product(4, 2100, 1100, 640)        # 256 x 256
    ffn(8, 8, 2, 256, 128)             # 16-row tiles
    ffn(4, 120, 2, 256, 256)           # 64 x 256
    ffn(4, 4100, 2, 256, 512)          # 256 x 256
    print("DEBUG CHILD OK", flush=True)


main()
