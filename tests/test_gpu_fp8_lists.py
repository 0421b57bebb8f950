"""Lists of several 256-row tiles per workgroup, every row against the definition in float64.

The gate/up kernel copies the next tile's gathered row numbers, scales and first blocks
behind the current tile; with more tiles than compute units every step of that runs.  All
tolerances stand in fp8_device_ref (narrow operands: the first product drops nothing).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_cases import flush
from oracle import permute as OP
from oracle import route as OR

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import fp8_device_ref as R  # noqa: E402
from test_gpu_fp8 import DEV, MARK, Layer  # noqa: E402


def _check_ffn(c: Layer, gateup_cut: bool) -> None:
    """Every row of the last run."""
    ids, _ = OR.route(c.logits_np, c.k)
    _, off, srt, _ = OP.permute(ids, c.E)
    x = torch.from_numpy(c.xv).to(DEV)
    rows = torch.from_numpy(np.asarray(srt, np.int64) // c.k).to(DEV)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    for e in range(c.E):
        lo, hi = int(off[e]), int(off[e + 1])
        if hi > lo:
            y, tol = R.ffn_rows(x[rows[lo:hi]], *(up(a) for a in c._parts[e]), gateup_cut)
            err = (c.layer.y_perm[lo:hi].double() - y).abs()
            bad = torch.nonzero(~(err <= tol))
            assert not len(bad), (e, bad[:4].tolist(), len(bad))


def _gateup_tiles(c: Layer) -> int:
    n = np.bincount(np.asarray(OR.route(c.logits_np, c.k)[0]).ravel(), minlength=c.E)
    return int(sum(-(-int(v) // 256) for v in n)) * (c.I // 128)


@pytest.mark.parametrize("T,H,I,E,k,zipf", [
    (4100, 256, 1280, 8, 4, None), (4100, 256, 1280, 8, 4, 1.5), (4096, 256, 1024, 64, 8, None),
    (4100, 384, 1280, 8, 4, None), (4100, 512, 1280, 8, 4, 1.0), (4100, 640, 1280, 8, 4, 1.0),
    (4100, 2048, 1280, 8, 4, None)])
def test_ffn_several_tiles_per_unit(T, H, I, E, k, zipf):
    """K of 2, 3, 4, 5 and 16 blocks, more gate/up tiles than twice the units."""
    flush(f"[ffn fp8 lists] T={T} H={H} I={I} E={E} k={k} zipf={zipf}")
    c = Layer(T, H, I, E, k, seed=T + H + E, zipf=zipf)
    assert _gateup_tiles(c) > 600
    y = c.run()
    _check_ffn(c, gateup_cut=False)
    ref = y.clone()
    assert torch.equal(c.run(), ref)
    assert bool((ref != MARK).any(1).all())


@pytest.mark.parametrize("T,H,I,E,k,zipf", [
    (4100, 256, 512, 4, 2, None), (4096, 512, 384, 8, 4, 1.4), (4100, 1024, 1280, 8, 4, 1.0),
    (2100, 2048, 1408, 6, 4, None)])
def test_ffn_tiles_on_ordinary_values(T, H, I, E, k, zipf):
    """Normal x and codes over the range, whose products the E4M3 MFMA cuts: gate and up sums
    within its bound, every row."""
    flush(f"[ffn fp8 lists, wide] T={T} H={H} I={I} E={E} k={k}")
    c = Layer(T, H, I, E, k, seed=T + H + 1, zipf=zipf, wide=True)
    assert _gateup_tiles(c) > 128
    c.run()
    _check_ffn(c, gateup_cut=True)
