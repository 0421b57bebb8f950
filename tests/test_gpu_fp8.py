"""moe_fp8_quantize, moe_fp8_matmul and moe_expert_ffn_fp8 against the float64 oracle.

Tolerances.  Quantisation: none, codes and scales are exact.  Product: with
eps = 2^-24 and mag = the sum of the magnitudes of an output's terms, a block's
128 products are added by the MFMA in fp32 (each addition off by at most one
ulp, 2 eps, whatever its rounding), then scaled (the product of the two scales
1, the multiply-add 1) and added over kb blocks (and up to 16 partial sums):
(2*128 + kb + 20) eps mag; the result is rounded to bf16 once, 2^-8 |y|.
To this comes what the instruction drops within its groups of 8 products
(O8.mfma_cut).  That property was read off the instruction, for the 16x16x128,
32x32x64 and 16x16x32 shapes alike: 2^16 - 2^16 + s gives s cut toward zero to
a multiple of 2^3 where the three share an aligned group of 8 consecutive k, and s
itself otherwise, whatever the accumulator holds.  By arithmetic: with the
largest product in [2^E, 2^(E+1)), each other product of the group loses less than
2^(E-13), seven of them less than 7 * 2^-13 of the largest; the largest itself
has at most 8 significant bits and loses nothing.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import synth
from gpu_cases import Case, flush
from oracle import ffn as OFF
from oracle import formats as OF
from oracle import fp8 as O8
from oracle import permute as OP
from oracle import route as OR

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_expert_ffn_router_amd as moe  # noqa: E402

DEV = torch.device("cuda")
EPS = 2.0 ** -24
MARK = 77.0


def _bf16(a):
    """numpy float -> (device bf16 tensor, its values in float64)."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16)
    return t.to(DEV), t.double().numpy()


# ---- quantisation ----------------------------------------------------------
def _quantize(x):
    T, K = x.shape
    codes = torch.full((T, K), 0xee, dtype=torch.uint8, device=DEV)
    scales = torch.full((T, -(-K // 128)), MARK, device=DEV)
    moe.moe_fp8_quantize(x, codes, scales)
    torch.cuda.synchronize()
    return codes.cpu().numpy(), scales.cpu().numpy()


@pytest.mark.parametrize("T,K", [(1, 8), (1, 128), (3, 136), (2, 1024), (17, 200), (5, 4096),
                                 (300, 72), (1025, 512), (1, 65536)])
def test_quantize_bit_exact(T, K):
    flush(f"[quantize] T={T} K={K}")
    rng = np.random.default_rng(T * 1000 + K)
    v = rng.normal(size=(T, K)) * np.exp(3 * rng.normal(size=(T, K)))
    v[:, rng.integers(0, K, 3)] = 0.0
    v[T // 2] = 0.0
    x, xv = _bf16(v)
    codes, scales = _quantize(x)
    rc, rs = O8.quantize(xv)
    assert np.array_equal(scales, rs.astype(np.float32))
    assert np.array_equal(codes, rc)


def test_quantize_every_bf16_magnitude():
    """Every finite bf16 as a block's maximum, beside a value of each size below it."""
    mag = np.arange(0x7f80, dtype=np.uint16)
    bits = np.zeros((len(mag), 128), np.uint16)
    bits[:, 0] = mag
    for j in range(1, 128):                    # smaller values of both signs
        bits[:, j] = np.maximum(mag.astype(np.int64) - 37 * j, 0).astype(np.uint16) | ((j & 1) << 15)
    x = torch.from_numpy(bits.view(np.int16)).to(DEV).view(torch.bfloat16)
    codes, scales = _quantize(x)
    step = 61                                  # the oracle is slow: every 61st magnitude, and the ends
    rows = np.unique(np.concatenate([np.arange(0, len(mag), step), np.arange(12),
                                     np.arange(len(mag) - 12, len(mag))]))
    rc, rs = O8.quantize(OF.bf16_value(bits[rows]))
    assert np.array_equal(scales[rows], rs.astype(np.float32))
    # -0.0 keeps its sign bit on both sides
    assert np.array_equal(codes[rows], rc)


def test_quantize_non_finite_blocks():
    v = np.ones((4, 384))
    x, _ = _bf16(v)
    x[0, 5], x[1, 130], x[2, 383], x[3, 0] = (float("inf"), float("nan"), float("-inf"), 448.0)
    codes, scales = _quantize(x)
    bad = np.isnan(scales)
    assert bad.tolist() == [[True, False, False], [False, True, False], [False, False, True],
                            [False] * 3]
    for t in range(4):
        for b in range(3):
            blk = codes[t, b * 128:(b + 1) * 128]
            assert np.all(blk == 0x7f) if bad[t, b] else np.all(blk != 0x7f)


# ---- product ---------------------------------------------------------------
def _codes(rng, shape):
    """E4M3 codes of normal values; a few at the ends of the range."""
    t = torch.from_numpy(rng.normal(size=shape) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
    c = t.view(torch.uint8).numpy().copy()
    c.reshape(-1)[rng.integers(0, c.size, max(1, c.size // 50))] = 0x7e   # 448
    c.reshape(-1)[rng.integers(0, c.size, max(1, c.size // 50))] = 0x81   # -2^-9
    return c


class Product:
    def __init__(self, M, N, K, E=0, counts=None, seed=0):
        rng = np.random.default_rng(seed)
        kb, nb = -(-K // 128), -(-N // 128)
        lead = (E,) if E else ()
        self.M, self.N, self.K, self.E = M, N, K, E
        self.a, self.w = _codes(rng, (M, K)), _codes(rng, lead + (N, K))
        self.sa = (np.exp(rng.normal(size=(M, kb))) * 0.01).astype(np.float32)
        self.sw = (np.exp(rng.normal(size=lead + (nb, kb))) * 0.01).astype(np.float32)
        self.counts = self.offsets = None
        if E:
            c = np.asarray(counts, np.int32)
            self.counts = c
            self.offsets = np.concatenate([[0], np.cumsum(c)]).astype(np.int32)

    def upload(self):
        up = lambda a: None if a is None else torch.from_numpy(a).to(DEV)  # noqa: E731
        self.d = [up(self.a), up(self.sa), up(self.w), up(self.sw)]
        self.c, self.o = up(self.counts), up(self.offsets)
        self.y = torch.full((self.M, self.N), MARK, dtype=torch.bfloat16, device=DEV)
        n = moe.moe_fp8_matmul_workspace(self.M, self.N, self.K, max(self.E, 1))
        self.ws = torch.full((n,), 0xff, dtype=torch.uint8, device=DEV) if n else None
        return self

    def call(self, stream=None):
        moe.moe_fp8_matmul(*self.d, self.y, self.ws, self.c, self.o, stream)

    def reference(self):
        """(y, tol): rows of no segment hold the mark, with no tolerance."""
        kb = -(-self.K // 128)

        def one(a, sa, w, sw):
            y, mag = O8.matmul(a, sa, w, sw)
            return y, (2.0 ** -8 * np.abs(y) + (1 + 2.0 ** -8) *
                       ((2 * 128 + kb + 20) * EPS * mag + O8.mfma_cut(a, sa, w, sw)))

        if not self.E:
            return one(self.a, self.sa, self.w, self.sw)
        y, tol = np.full((self.M, self.N), MARK), np.zeros((self.M, self.N))
        for e in range(self.E):
            lo, n = self.offsets[e], self.counts[e]
            if n:
                y[lo:lo + n], tol[lo:lo + n] = one(self.a[lo:lo + n], self.sa[lo:lo + n], self.w[e],
                                                   self.sw[e])
        return y, tol

    def check(self):
        y, tol = self.reference()
        got = self.y.double().cpu().numpy()
        bad = np.abs(got - y) > tol
        assert not bad.any(), (np.argwhere(bad)[:5], np.abs(got - y)[bad][:5])


DENSE = [  # M, N, K: single tokens, tile edges, odd columns, short last blocks on both sides
    (1, 1, 16), (1, 7168, 2048), (1, 130, 4096), (2, 16, 128), (15, 64, 256), (16, 65, 144),
    (17, 127, 1040), (33, 129, 272), (64, 256, 512), (65, 512, 384), (100, 1413, 2000),
    (128, 128, 128), (129, 257, 112), (200, 384, 640), (256, 256, 1024), (257, 511, 896),
    (300, 1000, 48), (513, 640, 256), (1000, 100, 2064), (5, 2048, 16384),
]


@pytest.mark.parametrize("M,N,K", DENSE)
def test_matmul_dense(M, N, K):
    flush(f"[matmul] M={M} N={N} K={K}")
    p = Product(M, N, K, seed=M + N + K).upload()
    p.call()
    torch.cuda.synchronize()
    p.check()


GROUPED = [  # E, counts, N, K, rows behind the last segment
    (1, [5], 64, 128, 0), (3, [0, 0, 0], 64, 128, 4), (4, [1, 0, 17, 3], 130, 256, 5),
    (5, [64, 65, 0, 63, 1], 256, 400, 0), (8, [0, 300, 2, 0, 0, 129, 128, 16], 384, 512, 9),
    (70, [i % 5 for i in range(70)], 96, 144, 1), (200, [1] * 200, 48, 128, 0),
    (2, [700, 260], 511, 272, 3), (1024, [3 if i % 100 == 0 else 0 for i in range(1024)], 32, 64, 2),
]


@pytest.mark.parametrize("E,counts,N,K,tail", GROUPED)
def test_matmul_grouped(E, counts, N, K, tail):
    M = sum(counts) + tail
    flush(f"[matmul] grouped E={E} M={M} N={N} K={K}")
    p = Product(M, N, K, E, counts, seed=E + N).upload()
    p.call()
    torch.cuda.synchronize()
    p.check()                                   # rows behind the last segment keep the mark


@pytest.mark.parametrize("M,N,K", [
    (33, 200, 2048), (40, 17, 1040), (100, 1, 272), (20, 4096, 144),       # 32 x 16 tiles
    (64, 4095, 1040), (65, 1301, 2064), (33, 4096, 16),                    # 32 x 32
    (128, 4096, 272), (250, 1413, 1168), (97, 3333, 2000),                 # 32 x 64
    (400, 1411, 400), (500, 1302, 144), (330, 2049, 640)])                 # 64 x 64, unaligned rows
def test_matmul_dozens_of_rows(M, N, K):
    """Tiles whose waves split K: fewer blocks than waves, a short last block, ragged edges."""
    flush(f"[matmul] M={M} N={N} K={K}")
    p = Product(M, N, K, seed=M + N + K).upload()
    p.call()
    torch.cuda.synchronize()
    p.check()
    ref = p.y.clone()
    p.y.fill_(MARK)
    p.call()
    torch.cuda.synchronize()
    assert torch.equal(p.y, ref)


@pytest.mark.parametrize("E,counts,N,K,tail", [
    (3, [20, 0, 33], 100, 1168, 2), (2, [0, 100], 1500, 400, 0), (4, [64, 1, 31, 32], 2050, 272, 3),
    (5, [0, 0, 60, 0, 0], 700, 1040, 7), (3, [900, 300, 101], 2501, 144, 5)])  # the last: 64 x 256
def test_matmul_dozens_of_rows_grouped(E, counts, N, K, tail):
    M = sum(counts) + tail
    flush(f"[matmul] grouped E={E} M={M} N={N} K={K}")
    p = Product(M, N, K, E, counts, seed=E + N).upload()
    p.call()
    torch.cuda.synchronize()
    p.check()


def test_matmul_extreme_scales():
    """Any fp32 scales: zero, subnormal, negative, large; a NaN code or scale reaches its row only."""
    p = Product(70, 160, 384, seed=3)
    p.sa[0], p.sa[1], p.sa[2] = 0.0, 1e-38, 1e30
    p.sa[3, 1], p.sw[0, 2] = -0.5, -2.0
    p.upload()
    p.d[0][5, 200] = 0x7f
    p.d[1][6, 0] = float("nan")
    p.call()
    torch.cuda.synchronize()
    got = p.y.double().cpu().numpy()
    assert np.all(np.isnan(got[5:7])) and np.all(np.isfinite(np.delete(got, [5, 6], 0)))
    y, tol = p.reference()
    tol = tol + 2.0 ** -126
    keep = np.delete(np.arange(70), [5, 6])
    assert np.all(np.abs(got - y)[keep] <= tol[keep])


def test_matmul_rows_do_not_depend_on_the_batch():
    """A row's result is the same bits alone, in a small batch and in a large one where the
    kernel is the same; repeated calls and other streams repeat the bits."""
    p = Product(300, 256, 512, seed=8).upload()
    p.call()
    torch.cuda.synchronize()
    ref = p.y.clone()
    for s in (None, torch.cuda.Stream()):
        p.y.fill_(MARK)
        torch.cuda.synchronize()
        p.call(s)
        torch.cuda.synchronize()
        assert torch.equal(p.y, ref)
    p.check()


def test_matmul_typed_codes():
    p = Product(20, 64, 128, seed=9).upload()
    p.d[0], p.d[2] = p.d[0].view(torch.float8_e4m3fn), p.d[2].view(torch.float8_e4m3fn)
    p.call()
    torch.cuda.synchronize()
    p.check()


def test_quantize_then_matmul_captured():
    """As used: quantise and product in one graph, replayed on new rows with eager work between."""
    T, N, K = 40, 256, 384
    p = Product(T, N, K, seed=10).upload()
    x = torch.zeros(T, K, dtype=torch.bfloat16, device=DEV)

    def step():
        moe.moe_fp8_quantize(x, p.d[0], p.d[1])
        p.call()

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for rep in range(3):
        t, v = _bf16(np.random.default_rng(rep).normal(size=(T, K)))
        x.copy_(t)
        p.y.fill_(MARK)
        g.replay()
        torch.cuda.synchronize()
        p.a, s = O8.quantize(v)
        p.sa = s.astype(np.float32)
        assert np.array_equal(p.d[0].cpu().numpy(), p.a)
        p.check()


def test_matmul_binding_refusals():
    p = Product(8, 32, 64).upload()
    a, sa, w, sw = p.d
    for args in ((a.float(), sa, w, sw, p.y), (a, sa[:4], w, sw, p.y), (a, sa, w[:, :32], sw, p.y),
                 (a, sa, w, sw.double(), p.y), (a, sa, w, sw, p.y[:, :16]), (a, sa, w, sw, p.y.float()),
                 (a, sa, w.cpu(), sw, p.y), (a.t(), sa, w, sw, p.y)):
        with pytest.raises(ValueError):
            moe.moe_fp8_matmul(*args)
    with pytest.raises(moe.MoeError):
        moe.moe_fp8_matmul(a, sa, w.view(2, 16, 64), torch.ones(2, device=DEV), p.y[:, :16].contiguous())


# ---- the expert FFN --------------------------------------------------------
# Rows x and gate/up codes take three neighbouring binades (Narrow below), so that the
# first product's groups of 8 lose nothing: their products are multiples of 2^-6 of
# the smallest binade's product and below 2^6 of it, 12 bits.  What is left of the first
# product's error is its fp32 additions, and h rounds to the definition's code
# except where it is that close to a border.
def _narrow(rng, shape):
    return (rng.choice([-1.0, 1.0], shape) * (1 + rng.integers(0, 8, shape) / 8)
            * 2.0 ** rng.integers(0, 3, shape))


def _ffn_reference(x, k, offsets, sorted_idx, parts, H, I):
    """(y, tol): the definition in float64 on bf16 rows x, and the tolerance.  Besides the
    products' own errors (as above), h may round to another code where it is closer to a code's
    border than its own error; such an element is off by what its interval spans."""
    X = O8.rows_value(*O8.quantize(x))
    A = int(offsets[-1])
    y, tol = np.zeros((A, H)), np.zeros((A, H))
    for e in range(len(offsets) - 1):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi <= lo:
            continue
        rows = X[np.asarray(sorted_idx[lo:hi]) // k]
        c13, s13, c2, s2 = parts(e)
        W13, W2 = O8.weight_value(c13, s13), O8.weight_value(c2, s2)
        c = (2 * 128 + H // 128 + 20) * EPS
        gu, dgu = rows @ W13.T, c * (np.abs(rows) @ np.abs(W13).T)
        g, u, dg, du = gu[:, :I], gu[:, I:], dgu[:, :I], dgu[:, I:]
        act = OFF.silu(g)
        h = act * u
        # |silu'| <= 1.1; 2^x and 1/x of one ulp, a sum and two products: 8 roundings; the
        # exponent's product with log2(e) and that constant: e^-g off by 2 |g| eps
        dh = (1.1 * dg * np.abs(u) + np.abs(act) * du + 1.1 * dg * du
              + (8 + 2 * np.abs(g)) * EPS * np.abs(h))
        hc, hs = O8.quantize(h)
        hq = O8.rows_value(hc, hs)
        off = np.zeros_like(h)
        for b in range(I // 128):
            s = slice(b * 128, (b + 1) * 128)
            am = np.abs(h[:, s])
            lo_m = np.max(np.maximum(am - dh[:, s], 0), axis=1)
            hi_m = np.max(am + dh[:, s], axis=1)
            for r in range(h.shape[0]):
                vals = [O8.decode(O8._round_codes(np.clip(v / q, -448, 448))) * q
                        for q in {O8.scale_of(lo_m[r]), O8.scale_of(hi_m[r])}
                        for v in (h[r, s] - dh[r, s], h[r, s] + dh[r, s])]
                vals.append(hq[r, s])
                off[r, s] = np.max(vals, axis=0) - np.min(vals, axis=0)
        y[lo:hi] = hq @ W2.T
        mag = (np.abs(hq) + off) @ np.abs(W2).T
        tol[lo:hi] = (2.0 ** -8 * np.abs(y[lo:hi]) + (1 + 2.0 ** -8) *
                      ((2 * 128 + I // 128 + 20) * EPS * mag + off @ np.abs(W2).T
                       + O8.mfma_cut(hc, hs, c2, s2)))
    return y, tol


class Layer:
    """A layer of FP8 records (narrow gate/up codes, any down codes), its batch and helper."""

    def __init__(self, T, H, I, E, k, seed, zipf=None, T_max=None, wide=False):
        rng = np.random.default_rng(seed)
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        wl = synth.Workload(f"fp8_{seed}", T=T, H=H, E=E, I=I, k=k, fmt="fp8_b128", seed=seed,
                            zipf=zipf)
        self.wl = wl
        self.logits_np = synth.make_logits(wl)
        self.logits = torch.from_numpy(self.logits_np).to(DEV)
        self.x, self.xv = _bf16(rng.normal(size=(T, H)) if wide else _narrow(rng, (T, H)))
        lay = synth.record_layout("fp8_b128", H, I)
        rec = np.zeros((E, lay["stride"]), np.uint8)
        self._parts = []
        for e in range(E):
            v13 = np.clip(rng.normal(size=(2 * I, H)) * 40, -448, 448) / 8
            c13 = (torch.from_numpy(v13 if wide else _narrow(rng, (2 * I, H))).to(torch.float8_e4m3fn)
                   .view(torch.uint8).numpy())
            c2 = _codes(rng, (H, I))
            s13 = (0.02 * (0.5 + rng.random((2 * I // 128, H // 128))) / np.sqrt(H)).astype(np.float32)
            s2 = (0.02 * (0.5 + rng.random((H // 128, I // 128)))).astype(np.float32)
            for name, v in (("w13", c13), ("w13s", s13), ("w2", c2), ("w2s", s2)):
                o, n = lay["sections"][name]
                rec[e, o:o + n] = np.ascontiguousarray(v).view(np.uint8).reshape(-1)
            self._parts.append((c13, s13, c2, s2))
        self.records = torch.from_numpy(rec).to(DEV)
        self.layer = moe.MoELayer("fp8_b128", E, H, I, k, T_max or T, lay["stride"])

    def run(self, base=None, slots=None):
        self.layer.route_permute(self.logits)
        self.layer.y_perm.fill_(MARK)
        W = self.layer.weights(self.records if base is None else base)
        self.layer.expert_ffn(W, self.x, self.T, slots, "fp8")
        torch.cuda.synchronize()
        return self.layer.y_perm

    def check(self):
        ids, _ = OR.route(self.logits_np, self.k)
        _, off, srt, _ = OP.permute(ids, self.E)
        y, tol = _ffn_reference(self.xv, self.k, off, srt, lambda e: self._parts[e], self.H, self.I)
        got = self.layer.y_perm[:self.T * self.k].double().cpu().numpy()
        bad = np.abs(got - y) > tol
        assert not bad.any(), (np.argwhere(bad)[:4], np.abs(got - y)[bad][:4], tol[bad][:4])


@pytest.mark.parametrize("T,H,I,E,k,zipf", [
    (1, 128, 128, 4, 2, None), (8, 256, 128, 16, 4, None), (5, 384, 256, 1, 1, None),
    (40, 512, 384, 8, 2, 1.2), (150, 256, 256, 6, 3, 0.7), (64, 1024, 512, 40, 8, None),
    (300, 384, 640, 3, 2, None), (16, 2048, 512, 64, 8, None), (600, 256, 256, 4, 2, 1.5),
    # 32-row gate/up tiles: 16 columns (few tiles), 32 columns, one expert's rows over many tiles
    (40, 1024, 256, 4, 2, 1.5), (90, 1152, 512, 8, 4, None), (64, 1024, 128, 3, 3, None),
    (33, 2048, 128, 2, 1, None), (100, 1024, 640, 7, 2, 2.5)])
def test_expert_ffn_fp8(T, H, I, E, k, zipf):
    flush(f"[ffn fp8] T={T} H={H} I={I} E={E} k={k}")
    c = Layer(T, H, I, E, k, seed=T + H + I, zipf=zipf)
    c.run()
    c.check()


@pytest.mark.parametrize("T,H,I,E,k,zipf", [
    (1, 512, 128, 4, 2, None), (8, 2048, 512, 64, 8, None),      # 16-row tiles
    (40, 512, 384, 8, 2, 1.2), (150, 384, 256, 6, 4, None),      # 64 x 256 tiles
    (90, 2048, 256, 6, 4, None), (90, 1152, 512, 8, 4, 1.0)])    # 32-row tiles
def test_expert_ffn_fp8_of_few_rows_keeps_every_product(T, H, I, E, k, zipf):
    """Ordinary values, whose products span more than the E4M3 MFMA keeps: few rows take their
    gate/up products exactly, with the tolerance of fp32 additions."""
    flush(f"[ffn fp8, wide] T={T} H={H} I={I} E={E} k={k}")
    c = Layer(T, H, I, E, k, seed=T + H + I + 1, zipf=zipf, wide=True)
    c.run()
    c.check()


@pytest.mark.parametrize("H", [256, 1024])
def test_expert_ffn_fp8_through_a_slot_table_and_larger_buffers(H):
    c = Layer(30, H, 256, 12, 3, seed=77, T_max=50)
    perm = torch.randperm(c.E)
    pool = torch.empty_like(c.records)
    pool[perm.to(DEV)] = c.records              # record e in slot perm[e]
    y = c.run(pool, perm.to(torch.int32).to(DEV))
    c.check()
    assert torch.all(y[c.T * c.k:] == MARK)     # rows behind the batch stay


def test_layer_forward_fp8_variant_captured():
    """The whole layer with the fp8 variant, captured and replayed on three batches with eager
    work between; every replay equals the eager bits."""
    wl = synth.Workload("fp8_graph", T=70, H=512, E=16, I=256, k=4, fmt="fp8_b128", seed=81)
    case = Case(wl)
    layer = moe.MoELayer("fp8_b128", wl.E, wl.H, wl.I, wl.k, wl.T, case.stride)
    W = layer.weights(case.records)
    lg, x = case.logits.clone(), case.x.clone()
    layer.forward(lg, x, W, variant="fp8")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.forward(lg, x, W, variant="fp8")
    for rep in range(3):
        lg.copy_(torch.from_numpy(synth.make_logits(wl, rep)))
        x.copy_(torch.from_numpy(synth.make_x(wl, rep).view(np.int16)).view(torch.bfloat16))
        layer.y.fill_(MARK)
        g.replay()
        torch.cuda.synchronize()
        got = layer.y[:wl.T].clone()
        layer.y.fill_(MARK)
        ref = layer.forward(lg, x, W, variant="fp8").clone()
        torch.cuda.synchronize()
        assert torch.equal(got, ref)
        # against the bf16-activation path: E4M3 rounds each x and h by at most 2^-4 of it, and the
        # products' sums average those
        alt = layer.forward(lg, x, W, variant="prefill")
        torch.cuda.synchronize()
        rms = float((ref.float() - alt.float()).norm() / alt.float().norm())
        assert rms < 2.0 ** -4, rms


def test_expert_ffn_fp8_masked_rows_zero_and_nan():
    """A zero token gives zero rows; a token with a NaN gives NaN rows and no other."""
    c = Layer(20, 256, 128, 4, 2, seed=90)
    c.x[3] = 0
    c.x[7, 9] = float("nan")
    y = c.run().float().cpu().numpy()
    inv = c.layer.inv_idx[:c.T * c.k].cpu().numpy().reshape(c.T, c.k)
    assert np.all(y[inv[3]] == 0) and np.all(np.isnan(y[inv[7]]))
    assert np.all(np.isfinite(np.delete(y, inv[7], 0)))


@pytest.mark.parametrize("T,H,I", [(3, 256, 128), (20, 256, 128), (20, 1024, 128),
                                   (2100, 256, 512)])  # tiles of 16, 64, 32 and 256 rows
def test_expert_ffn_fp8_nan_weight_code(T, H, I):
    """A NaN code among an expert's gate, up or down weights: NaN where its rows meet it, and
    nowhere else."""
    for name, n, whole in (("w13", 5 * H + 9, True), ("w13", (I + 7) * H, True),
                           ("w2", 3 * I + 2, False)):
        c = Layer(T, H, I, 4, 2, seed=91)
        o, _ = synth.record_layout("fp8_b128", H, I)["sections"][name]
        c.records[1, o + n] = 0x7f
        y = c.run()[:T * 2].float().cpu().numpy()
        ids, _ = OR.route(c.logits_np, 2)
        _, off, _, _ = OP.permute(ids, 4)
        bad = np.zeros_like(y, bool)
        bad[off[1]:off[2], slice(None) if whole else 3] = True
        assert np.array_equal(np.isnan(y), bad)


# ---- every kernel the size rules choose ------------------------------------
def _check_all_rows(p, sample):
    """Every output against the product in float64 on the device, within a bound that only a
    misplaced, dropped or doubled term can pass; the sampled rows against the oracle's bound.

    The crude bound: with at most one subnormal operand the product of the binades is at most 8
    times the product itself, so a group's largest (mfma_cut's `top`) is at most 8 times the
    group's magnitude sum; a pair of two subnormals has 2^-12, no more than any pair of normal
    codes beside it.  Summed over the groups: 7 * 2^-13 * 8 mag."""
    kb = -(-p.K // 128)
    A = p.d[0].view(torch.float8_e4m3fn).double() * p.d[1].double().repeat_interleave(128, 1)[:, :p.K]
    w, sw = p.d[2].view(torch.float8_e4m3fn), p.d[3].double()
    segs = [(0, p.M, 0)] if not p.E else [(int(p.offsets[e]), int(p.offsets[e] + p.counts[e]), e)
                                         for e in range(p.E) if p.counts[e]]
    seen = torch.zeros(p.M, dtype=torch.bool, device=DEV)
    for lo, hi, e in segs:
        we, se = (w[e], sw[e]) if p.E else (w, sw)
        W = we.double() * se.repeat_interleave(128, 0)[:p.N].repeat_interleave(128, 1)[:, :p.K]
        y, mag = A[lo:hi] @ W.t(), A[lo:hi].abs() @ W.t().abs()
        err = (p.y[lo:hi].double() - y).abs()
        tol = 2.0 ** -8 * y.abs() + (7 * 2.0 ** -13 * 8 + (256 + kb + 20) * EPS) * mag
        assert bool((err <= tol).all()), (e, torch.nonzero(err > tol)[:4].tolist())
        seen[lo:hi] = True
    assert bool((p.y[~seen] == MARK).all())
    got = p.y.double().cpu().numpy()
    for lo, hi, e in segs:
        rows = [r for r in sample if lo <= r < hi]
        if rows:
            we, se = (p.w[e], p.sw[e]) if p.E else (p.w, p.sw)
            y, mag = O8.matmul(p.a[rows], p.sa[rows], we, se)
            tol = (2.0 ** -8 * np.abs(y) + (1 + 2.0 ** -8) *
                   ((256 + kb + 20) * EPS * mag + O8.mfma_cut(p.a[rows], p.sa[rows], we, se)))
            assert np.all(np.abs(got[rows] - y) <= tol)


@pytest.mark.parametrize("M,N,K", [
    (1100, 2500, 128), (1100, 2500, 272), (1100, 2500, 1040),              # 64 x 256 tiles
    (8200, 2300, 144), (8200, 2300, 272), (8200, 2300, 384), (8200, 2300, 400),
    (8200, 2300, 640), (8200, 2300, 1040), (16400, 2050, 512),             # 256 x 256, several a unit
    (33, 65536, 16), (40, 48, 65536), (3, 33, 65536)])
def test_matmul_tiles(M, N, K):
    flush(f"[matmul tiles] M={M} N={N} K={K}")
    p = Product(M, N, K, seed=M + K).upload()
    p.call()
    torch.cuda.synchronize()
    _check_all_rows(p, sorted({0, M // 2, M - 1, min(M - 1, 8192)}))
    ref = p.y.clone()
    for s in (None, torch.cuda.Stream()):                                  # the same bits again
        p.y.fill_(MARK)
        torch.cuda.synchronize()
        p.call(s)
        torch.cuda.synchronize()
        assert torch.equal(p.y, ref)


@pytest.mark.parametrize("E,counts,N,K,tail", [
    (6, [2000, 1, 0, 129, 128, 900], 1500, 640, 5), (3, [0, 4097, 30], 2048, 400, 0),
    (16, [700, 3, 255, 256, 257, 0, 1500, 128, 129, 64, 65, 900, 1, 0, 511, 513], 1000, 272, 11),
    (40, [60 + 7 * i for i in range(40)], 600, 512, 3), (9, [40, 64, 65, 0, 1, 128, 80, 70, 33], 3200, 1040, 2),
    (300, [i % 23 for i in range(300)], 512, 256, 0), (300, [(i * 7) % 90 for i in range(300)], 700, 144, 1)])
def test_matmul_grouped_tiles(E, counts, N, K, tail):
    M = sum(counts) + tail
    flush(f"[matmul tiles] grouped E={E} M={M} N={N} K={K}")
    p = Product(M, N, K, E, counts, seed=E + K).upload()
    p.call()
    torch.cuda.synchronize()
    off = p.offsets
    _check_all_rows(p, sorted({int(r) for e in range(0, E, max(1, E // 6))
                               for r in (off[e], off[e + 1] - 1) if 0 <= r < M - tail}))


@pytest.mark.parametrize("T,H,I,E,k,zipf", [(4100, 256, 512, 4, 2, None), (2100, 384, 640, 5, 4, 1.0),
                                            (4096, 512, 384, 8, 4, 1.4)])
def test_expert_ffn_fp8_tiles(T, H, I, E, k, zipf):
    """The 256-row gate/up tiles: sampled tokens' rows against the definition."""
    flush(f"[ffn fp8 tiles] T={T} H={H} I={I} E={E} k={k}")
    c = Layer(T, H, I, E, k, seed=T + I, zipf=zipf)
    y = c.run()
    ids, _ = OR.route(c.logits_np, k)
    _, off, srt, _ = OP.permute(ids, E)
    got = y[:T * k].double().cpu().numpy()
    assert np.all(np.isfinite(got))
    for e in range(E):                       # each expert's first, last and a few other rows
        lo, hi = int(off[e]), int(off[e + 1])
        if hi <= lo:
            continue
        rows = sorted({lo, hi - 1, (lo + hi) // 2, min(hi - 1, lo + 255), min(hi - 1, lo + 256),
                       max(lo, hi - 130)})
        sub = np.concatenate([[0] * (e + 1), [len(rows)] * (E - e)])
        yy, tol = _ffn_reference(c.xv, k, sub, np.asarray(srt)[rows], lambda q: c._parts[q], H, I)
        assert np.all(np.abs(got[rows] - yy) <= tol), e


def test_two_products_at_once():
    """Two products on two streams at the same time: each with the bits it has alone."""
    ps = [Product(M, 2300, 640, seed=M).upload() for M in (8200, 7000)]
    refs = []
    for p in ps:
        p.call()
        torch.cuda.synchronize()
        refs.append(p.y.clone())
        p.y.fill_(MARK)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for p, s in zip(ps, streams):
            p.call(s)
    torch.cuda.synchronize()
    for p, r in zip(ps, refs):
        assert torch.equal(p.y, r)
