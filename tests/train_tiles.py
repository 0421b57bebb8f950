"""Which tiles the expert training calls take, by the rule of csrc/expert_train.hip over the source's own
constants: so that a test can say which kernels it runs."""
from __future__ import annotations

import os
import re

from conftest import ROOT

_SRC = open(os.path.join(ROOT, "moe_expert_ffn_router_amd", "csrc", "expert_train.hip")).read()


def _const(name: str) -> int:
    return int(re.search(rf"\b{name} = (\d+)[,;]", _SRC).group(1))


ROW256, ROW128, W256, W128 = map(_const, ("kRowTiles256", "kRowTiles128", "kWeightTiles256", "kWeightTiles128"))
ROWS256, ROWS128 = _const("kRows256"), _const("kRows128")
TWO_ROWS, TWO_VALUES = _const("kTwoRows"), _const("kTwoValues")


def sides(E: int, H: int, I: int, A: int) -> dict:
    """Side of the tiles of each product of A rows (T * k) over E experts of H x I."""
    up = lambda a, b: -(-a // b)  # noqa: E731
    two = A <= min(TWO_ROWS, TWO_VALUES // I)
    touched = min(A, E)

    def rows(n):
        about = lambda s: (A // s + (touched + 1) // 2) * up(n, s)  # noqa: E731
        if not two and about(256) >= ROW256 and A > ROWS256 * touched:
            return 256
        return 128 if not two and about(128) >= ROW128 and A >= ROWS128 * touched else 64

    def weights(m, n):
        tiles = lambda s: E * up(m, s) * up(n, s)  # noqa: E731
        if tiles(256) >= W256 and not two:
            return 256
        return 128 if tiles(128) >= W128 else 64

    return {"gate_up": rows(2 * I), "down": rows(H), "dh": rows(I), "dx": rows(H),
            "w13": weights(2 * I, H), "w2": weights(H, I)}
