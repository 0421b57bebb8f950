"""The float64 device form of the FP8 definitions against the oracle (on the CPU)."""
from __future__ import annotations

import numpy as np
import torch

import fp8_device_ref as R
from oracle import fp8 as O8


def test_quantize_is_the_oracles():
    rng = np.random.default_rng(1)
    v = rng.normal(size=(9, 384)) * np.exp(4 * rng.normal(size=(9, 384)))
    v[3, :128], v[4, 7], v[5, 9], v[6, 200] = 0.0, 448.0, 448.0 * 2.0 ** 9, 2.0 ** -130
    c, s = O8.quantize(v)
    got, gs = R.quantize(torch.from_numpy(v))
    assert np.array_equal(gs.numpy()[:, ::128], s) and np.array_equal(got.numpy(), O8.rows_value(c, s))


def test_product_and_cut_are_the_oracles():
    rng = np.random.default_rng(2)
    M, N, K = 20, 150, 272
    a, w = (rng.integers(0, 254, s).astype(np.uint8) for s in ((M, K), (N, K)))
    a[a == 0x7f], w[w == 0x7f] = 0x7e, 0x7e                    # no NaN codes
    a[:, :40] &= 0x87                                          # a stretch of subnormals and zeros
    sa, sw = (rng.random(s).astype(np.float32) for s in ((M, 3), (2, 3)))
    y, mag = O8.matmul(a, sa, w, sw)
    cut = O8.mfma_cut(a, sa, w, sw)
    t = [torch.from_numpy(v) for v in (a, sa, w, sw)]
    got, tol = R.matmul(*t)
    base = R.matmul(*t, with_cut=False)[1]
    assert np.allclose(got.numpy(), y, rtol=0, atol=1e-12 * mag.max())
    c = ((tol - base) / (1 + 2.0 ** -8)).numpy()
    # never below the oracle's bound; above it only by raised subnormals
    assert np.all(c >= cut * (1 - 1e-9)) and np.all(c <= 2 * cut)
