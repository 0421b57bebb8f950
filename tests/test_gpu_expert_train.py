"""moe_expert_ffn_train and moe_expert_ffn_backward on the GPU against the formulas in 64 bits.

Tolerances, per element, from the roundings that the header names.  u = 2^-24, b = 2^-8 (half a
step of bf16), M(.) the same sum over magnitudes.  A product of K terms on the MFMA adds them
in fp32 in an order of its own: off by at most 2 K u M (each addition by one unit at most, not
half).  The sigmoid comes from the hardware's 2^x and 1/x: relative error (|g| + 8) 2^-23, and
2^-126 where it leaves the normal range.
  g, u     2 H u M + b |g|                                        (stored)
  h        1.1 |u| e_g + |silu(g)| e_u + (|g| + 8) 2^-22 |h| + b |h|   from the unrounded sums
  y        sum |Wd| e_h + 2 I u M + b |y|
  dh       2 H u M
  du       |silu| e_dh + (|g| + 8) 2^-22 |du| + b |du|
  dg       |u silu'| e_dh + (|g| + 8) 2^-22 |dh u| s (1 + 2 |g|) + b |dg|
  dx, dW   sum over the other operand's magnitudes of these + 2 K u M (+ b of a bf16 result)
These bounds add every rounding's worst case; besides, the 2-norm of the whole error is held
to what independent roundings give: each is at most b relative and uniform over its step, so
b / sqrt(3) of the result's norm, two of them in a row (operand and result) sqrt(2) of that; 1.5
times that is allowed for outputs of a thousand elements and more.
Batches of at most 96 rows and 32768 values of h keep h, dg and du in two parts: the first cut to bf16, what is left
below 2^-7 of it rounded to bf16, so 2^-15 stands for their b above (and one rounding less).
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from gpu_cases import flush

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_expert_ffn_router_amd as moe  # noqa: E402

DEV = torch.device("cuda")
BF, F32 = torch.bfloat16, torch.float32
U, B = 2.0 ** -24, 2.0 ** -8
MARK = 3.5


class Case:
    """Experts with the given numbers of rows, `behind` rows that belong to none; gathered: token
    rows through sorted_idx, else rows in expert order."""

    def __init__(self, counts, H, I, k=1, behind=0, gathered=True, seed=0, size=1.0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
        self.E, self.H, self.I, self.k = len(counts), H, I, k
        n = sum(counts) + behind
        self.T = -(-n // k)
        self.A = self.T * k
        self.n = sum(counts)
        E = self.E
        self.counts = torch.tensor(counts, dtype=torch.int32, device=DEV)
        self.ends = np.concatenate([[0], np.cumsum(counts)]).astype(int)
        self.offsets = torch.from_numpy(self.ends).int().to(DEV)
        self.sorted_idx = torch.randperm(self.A, generator=g, device=DEV).int() if gathered else None
        self.x = (rnd(self.T if gathered else self.A, H) * size).to(BF)
        self.rows = self.x[self.sorted_idx.long() // k] if gathered else self.x
        w13, w2 = (rnd(E, 2 * I, H) * H ** -0.5).to(BF), (rnd(E, H, I) * I ** -0.5).to(BF)
        self.rec = torch.cat([w13.view(E, -1), w2.view(E, -1)], 1).contiguous()
        self.w13, self.w2 = w13.double(), w2.double()
        self.W = moe.experts("bf16", E, H, I, self.rec, self.rec.shape[1] * 2)
        self.gu = (rnd(self.A, 2 * I) * 1.5 * size).to(BF)
        self.dy = (rnd(self.A, H) * 0.1).to(BF)
        self.ws = self.new(max(moe.moe_expert_ffn_backward_workspace(self.W, self.T, k), 256),
                           dtype=torch.uint8)

    def new(self, *shape, dtype=BF):
        return torch.full(shape, 255 if dtype is torch.uint8 else MARK, dtype=dtype, device=DEV)

    def forward(self, stream=None):
        gu, y = self.new(self.A, 2 * self.I), self.new(self.A, self.H)
        moe.moe_expert_ffn_train(self.W, self.x, self.T, self.k, self.counts, self.offsets,
                                 self.sorted_idx, gu, y, self.ws, stream=stream)
        return gu, y

    def backward(self, dtype=BF, accumulate=False, out=None, stream=None):
        E, H, I = self.E, self.H, self.I
        o = out or (self.new(self.A, H), self.new(E, 2 * I, H, dtype=dtype), self.new(E, H, I, dtype=dtype))
        moe.moe_expert_ffn_backward(self.W, self.x, self.T, self.k, self.counts, self.offsets,
                                    self.sorted_idx, self.gu, self.dy, self.ws, *o,
                                    accumulate=accumulate, stream=stream)
        return o


def close(got, want, tol, what, roundings=2):
    got = got.double()
    bad = ((got - want).abs() > tol) | got.isnan()
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[:4].tolist(),
                                 float(((got - want).abs() / tol.clamp(min=1e-300)).max()))
    if want.numel() >= 1000 and float(want.norm()) > 0:
        rel = float((got - want).norm() / want.norm())
        assert rel <= 1.5 * math.sqrt(roundings) * B / math.sqrt(3), (what, rel)


def two_parts(rows, I):
    return rows <= 96 and rows * I <= 32768


def check_forward(c, gu, y, rows=None):
    """rows: of the batch, where they are more than the case's."""
    I, H = c.I, c.H
    few = two_parts(rows or c.A, I)
    hb, roundings = (2.0 ** -15, 1) if few else (B, 2)
    for e in range(c.E):
        p = slice(c.ends[e], c.ends[e + 1])
        if p.start == p.stop:
            continue
        x, w13, w2 = c.rows[p].double(), c.w13[e], c.w2[e]
        z, zm = x @ w13.t(), x.abs() @ w13.abs().t()
        ez = 2 * H * U * zm
        close(gu[p], z, ez + B * z.abs(), f"gate_up {e}", 1)
        g, u = z[:, :I], z[:, I:]
        sg = torch.sigmoid(g) * g
        h = sg * u
        eh = 1.1 * u.abs() * ez[:, :I] + sg.abs() * ez[:, I:] + ((g.abs() + 8) * 2.0 ** -22 + hb) * h.abs()
        eh = eh + 2.0 ** -126 * (g * u).abs()
        want = h @ w2.t()
        tol = eh @ w2.abs().t() + 2 * I * U * (h.abs() @ w2.abs().t()) + B * want.abs()
        close(y[p], want, tol, f"y {e}", roundings)
    assert bool((gu[c.n:] == MARK).all()) and bool((y[c.n:] == MARK).all())


def check_backward(c, dx, d13, d2, base=0.0, rows=None):
    I, H = c.I, c.H
    few = two_parts(rows or c.A, I)
    hb, roundings = (2.0 ** -15, 1) if few else (B, 2)
    f32 = d13.dtype is F32
    r = 0.0 if f32 else B
    for e in range(c.E):
        p = slice(c.ends[e], c.ends[e + 1])
        n = p.stop - p.start
        x, w13, w2 = c.rows[p].double(), c.w13[e], c.w2[e]
        g, u, dy = c.gu[p, :I].double(), c.gu[p, I:].double(), c.dy[p].double()
        s = torch.sigmoid(g)
        sg, d = s * g, s * (1 + g * (1 - s))
        dh, edh = dy @ w2, 2 * H * U * (dy.abs() @ w2.abs())
        du, dg, h = dh * sg, dh * u * d, sg * u
        k22 = (g.abs() + 8) * 2.0 ** -22
        tiny = 2.0 ** -126 * (1 + g.abs()) * (1 + u.abs()) * (1 + dh.abs())
        edu = sg.abs() * edh + (k22 + hb) * du.abs() + tiny
        edg = (u * d).abs() * edh + k22 * (dh * u).abs() * s * (1 + 2 * g.abs()) + hb * dg.abs() + tiny
        eh = (k22 + hb) * h.abs() + tiny
        dz, edz = torch.cat([dg, du], 1), torch.cat([edg, edu], 1)
        if n:
            want = dz @ w13
            tol = edz @ w13.abs() + 4 * I * U * (dz.abs() @ w13.abs()) + B * want.abs()
            close(dx[p], want, tol, f"dx {e}", roundings)
        want = dz.t() @ x
        tol = edz.t() @ x.abs() + 2 * (n + 1) * U * (dz.abs().t() @ x.abs() + abs(base)) + r * want.abs()
        close(d13[e] - base, want, tol, f"d_w13 {e}", roundings)
        want = dy.t() @ h
        tol = dy.abs().t() @ eh + 2 * (n + 1) * U * (dy.abs().t() @ h.abs() + abs(base)) + r * want.abs()
        close(d2[e] - base, want, tol, f"d_w2 {e}", roundings)
        if n == 0:
            assert bool((d13[e] == base).all()) and bool((d2[e] == base).all())
    assert bool((dx[c.n:] == MARK).all())


# rows per expert around every tile and block size, experts without rows first, last and between
CASES = [
    dict(counts=[1], H=128, I=128),
    dict(counts=[0, 3], H=256, I=128, behind=2),
    dict(counts=[63, 0, 64, 65, 1, 0], H=128, I=256, k=2, behind=3),
    dict(counts=[127, 128, 129, 31, 33, 32], H=384, I=128, k=3),
    dict(counts=[0, 255, 256, 257, 2, 15, 17, 16], H=256, I=384, k=2, gathered=False),
    dict(counts=[511, 0, 513, 5], H=640, I=640, k=4, behind=9),
    dict(counts=[1300], H=512, I=256, k=1, gathered=False, behind=300),
    dict(counts=[3, 0, 1, 2] * 75, H=128, I=128, k=5, behind=1),
    dict(counts=[1] * 40, H=1152, I=128, k=8),
    dict(counts=[40, 700, 90], H=128, I=1152, k=16),
    dict(counts=[2, 200, 20], H=2048, I=512, k=2),
    dict(counts=[0, 0, 0], H=256, I=256, behind=7),
    dict(counts=[1] * 1024, H=128, I=128, k=2),
    # enough tiles of 256 x 256 for them to be taken: many blocks and few, columns past the last whole
    # tile, experts' rows in short and whole blocks, one expert with most of them
    dict(counts=[0, 700, 256, 257, 255, 1, 63, 64, 65, 0, 512, 640, 300, 128, 129, 191, 900, 31, 400, 33],
         H=1152, I=1152, k=2, behind=5),
    dict(counts=[3, 2900, 0, 1100, 17, 64], H=1024, I=1408, k=3, gathered=False, behind=2),
    dict(counts=[70, 66, 130, 0, 64, 100] * 21, H=128, I=2048, k=4),
    dict(counts=[70, 66, 130, 0, 64, 100] * 21, H=2048, I=128, k=1, gathered=False),
    dict(counts=[80] * 300, H=256, I=256, k=8),
    # for the tiles of 128 x 128: products over rows, over few rows an expert, of weights
    dict(counts=[0, 255, 256, 257, 129, 1, 511, 340, 250], H=2048, I=2048, k=2, behind=4),
    dict(counts=[40, 0, 17, 64, 63, 100] * 10, H=1024, I=640, k=3),
    dict(counts=[179, 128, 64, 300, 0, 1, 127, 400, 250, 65, 200, 129, 500], H=1024, I=384, k=3, behind=1),
    dict(counts=[179, 128, 64, 300, 0, 1, 127, 400, 250], H=640, I=640, gathered=False),
]
CASES += [
    dict(counts=[96], H=256, I=256),
    dict(counts=[97], H=256, I=256),
    dict(counts=[2, 83], H=256, I=384),
    dict(counts=[86], H=256, I=384, gathered=False),
    dict(counts=[129], H=256, I=384),
    dict(counts=[0, 20, 12, 0], H=1024, I=1024, k=2),
    dict(counts=[1], H=1152, I=16384),
    dict(counts=[1, 0, 2], H=512, I=1024, gathered=False),
    dict(counts=[65, 0, 31], H=128, I=128),
    dict(counts=[3, 0, 1, 0] * 8, H=2048, I=1024, k=4),
    dict(counts=[60, 4, 0, 32], H=4096, I=512, gathered=False),
]
IDS = [f"{len(c['counts'])}e{sum(c['counts'])}r{c['H']}x{c['I']}" for c in CASES]


@pytest.mark.parametrize("spec", CASES, ids=IDS)
def test_forward(spec):
    flush(f"[train] forward {spec['counts'][:8]} H={spec['H']} I={spec['I']}")
    c = Case(**spec)
    gu, y = c.forward()
    torch.cuda.synchronize()
    check_forward(c, gu, y)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("spec", CASES, ids=IDS)
def test_backward(spec, dtype):
    flush(f"[train] backward {spec['counts'][:8]} H={spec['H']} I={spec['I']} {dtype}")
    c = Case(**spec, seed=1)
    out = c.backward(dtype)
    torch.cuda.synchronize()
    check_backward(c, *out)


def test_accumulate():
    c = Case([5, 0, 300, 64], 256, 384, k=3, behind=1, seed=2)
    out = (c.new(c.A, c.H), torch.full((4, 768, 256), 0.25, device=DEV), torch.full((4, 256, 384), 0.25, device=DEV))
    c.backward(accumulate=True, out=out)
    check_backward(c, *out, base=0.25)
    alone = c.backward(F32)
    c.backward(accumulate=True, out=(out[0], *(t.clone() for t in alone[1:])))
    twice = (out[0], *(t.clone() for t in alone[1:]))
    c.backward(accumulate=True, out=twice)
    for a, t in zip(alone[1:], twice[1:]):
        assert torch.equal(2 * a, t)


def test_each_output_alone():
    c = Case([70, 1, 0, 130], 256, 256, k=2, seed=3)
    whole = c.backward()
    for i in range(3):
        out = [None, None, None]
        out[i] = torch.full_like(whole[i], MARK)
        c.backward(out=tuple(out))
        assert torch.equal(out[i], whole[i])
    c.backward(out=(None, None, None))


def test_no_rows_at_all():
    """T = 0: the weights' gradients become 0 (counts are not read); accumulated ones stay."""
    c = Case([4, 4], 128, 128, seed=4)
    d13, d2 = c.new(2, 256, 128), c.new(2, 128, 128)
    empty = c.x[:0]
    args = (c.W, c.x, 0, 1, c.counts, c.offsets, c.sorted_idx, c.gu, c.dy, c.ws)
    assert empty.numel() == 0
    moe.moe_expert_ffn_backward(*args, d_w13=d13, d_w2=d2)
    assert not d13.any() and not d2.any()
    f13, f2 = c.new(2, 256, 128, dtype=F32), c.new(2, 128, 128, dtype=F32)
    moe.moe_expert_ffn_backward(*args, d_w13=f13, d_w2=f2, accumulate=True)
    assert bool((f13 == MARK).all()) and bool((f2 == MARK).all())


def test_integers_are_exact():
    """Sums of small integers lose nothing: every product and place of the weights' gradients and of
    gate_up, bit by bit."""
    counts, H, I = [0, 77, 300, 64, 1], 384, 256
    c = Case(counts, H, I, k=2, seed=5)
    g = torch.Generator(device=DEV).manual_seed(6)
    c.x.copy_(torch.randint(-2, 3, c.x.shape, generator=g, device=DEV))
    c.rows = c.x[c.sorted_idx.long() // 2]
    rec = torch.randint(-1, 2, c.rec.shape, generator=g, device=DEV).to(BF)
    # sparse enough that the sums stay within bf16's 8 bits
    rec *= (torch.rand(c.rec.shape, generator=g, device=DEV) < 0.05)
    c.rec.copy_(rec)
    w13 = c.rec[:, :2 * I * H].view(5, 2 * I, H).double()
    gu, _ = c.forward()
    for e in range(5):
        p = slice(c.ends[e], c.ends[e + 1])
        want = c.rows[p].double() @ w13[e].t()
        assert bool((want.abs() <= 256).all()) and torch.equal(gu[p].double(), want)
    # dW2 = dy^T h with g = 64 (the sigmoid is 1): h = 64 u, an integer within 8 bits
    c.gu[:, :I] = 64.0
    c.gu[:, I:] = torch.randint(-2, 3, (c.A, I), generator=g, device=DEV).to(BF)
    c.dy.copy_(torch.randint(-3, 4, c.dy.shape, generator=g, device=DEV))
    _, _, d2 = c.backward(F32)
    for e in range(5):
        p = slice(c.ends[e], c.ends[e + 1])
        assert torch.equal(d2[e].double(), c.dy[p].double().t() @ (64.0 * c.gu[p, I:].double()))


def test_rows_that_are_not_finite():
    """NaN and infinite rows behind the last segment, or of another expert, reach no result."""
    c = Case([33, 65, 0, 7], 256, 128, k=1, behind=40, seed=7)
    dx, d13, d2 = c.backward(F32)
    gu, y = c.forward()
    bad = c.sorted_idx[c.n:].long()
    c.x[bad], c.gu[c.n:], c.dy[c.n:] = float("nan"), float("inf"), float("nan")
    again = c.backward(F32)
    gu2, y2 = c.forward()
    for a, b in ((dx, again[0]), (d13, again[1]), (d2, again[2]), (gu, gu2), (y, y2)):
        assert torch.equal(a[:c.n] if a.shape[0] == c.A else a, b[:c.n] if b.shape[0] == c.A else b)
    c.dy[40] = float("nan")      # a row of expert 1
    dx3, d133, d23 = c.backward(F32)
    assert bool(dx3[40].isnan().all()) and not bool(dx3[:40].isnan().any()) and not bool(dx3[41:98].isnan().any())
    assert bool(d23[1].isnan().all()) and not bool(d23[[0, 2, 3]].isnan().any())
    assert bool(d133[1].isnan().any()) and not bool(d133[[0, 2, 3]].isnan().any())


def test_large_gates():
    """Gates far out on both sides: the sigmoid's ends, without NaN."""
    c = Case([64, 30], 128, 128, seed=8)
    c.gu[:, :64] = torch.linspace(-200, 200, 64, device=DEV).to(BF)
    out = c.backward(F32)
    assert not any(bool(t[:c.n].isnan().any()) for t in out)
    check_backward(c, *out)


def test_gradients_are_differences():
    """The whole chain against central differences of the 64-bit forward along random directions."""
    c = Case([20, 44], 256, 128, k=1, gathered=False, seed=9, size=0.5)
    gu, y = c.forward()
    c.gu = gu
    dx, d13, d2 = c.backward(F32)

    def loss(x, w13, w2):
        t = 0.0
        for e in range(2):
            p = slice(c.ends[e], c.ends[e + 1])
            z = x[p] @ w13[e].t()
            h = z[:, :c.I] * torch.sigmoid(z[:, :c.I]) * z[:, c.I:]
            t = t + ((h @ w2[e].t()) * c.dy[p].double()).sum()
        return float(t)

    g = torch.Generator(device=DEV).manual_seed(10)
    ops = [c.x.double(), c.w13, c.w2]
    for i, grad in enumerate((dx, d13, d2)):
        v = torch.randn(ops[i].shape, generator=g, device=DEV, dtype=torch.float64)
        step = 1e-4
        up, dn = list(ops), list(ops)
        up[i], dn[i] = ops[i] + step * v, ops[i] - step * v
        want = (loss(*up) - loss(*dn)) / (2 * step)
        # the direction's share of the gradient's error: independent roundings of about 3 b / sqrt(3)
        # relative each, so 5 standard deviations of their sum
        tol = 5 * 3 * B / math.sqrt(3) * float((grad.double() * v).norm()) + 1e-5 * abs(want)
        assert abs(float((grad.double() * v).sum()) - want) <= tol


def test_repeat_stream_and_graph():
    c = Case([100, 0, 257, 31], 384, 256, k=2, behind=2, seed=11)
    gu, y = c.forward()
    first = c.backward()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, c.backward()))
        assert all(torch.equal(a, b) for a, b in zip((gu, y), c.forward()))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        got = c.backward(stream=s)
        f = c.forward(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, got)) and torch.equal(f[1], y)
    # captured: the batch changes between replays, its row counts too
    graph = torch.cuda.CUDAGraph()
    out = c.backward()
    torch.cuda.synchronize()
    fo = (c.new(c.A, 2 * c.I), c.new(c.A, c.H))
    with torch.cuda.graph(graph):
        moe.moe_expert_ffn_train(c.W, c.x, c.T, c.k, c.counts, c.offsets, c.sorted_idx, *fo, c.ws)
        c.backward(out=out)
    for r, counts in enumerate(([100, 0, 257, 31], [0, 388, 0, 0], [97, 97, 97, 97])):
        c.counts.copy_(torch.tensor(counts, dtype=torch.int32))
        c.offsets.copy_(torch.tensor([0] + np.cumsum(counts).tolist(), dtype=torch.int32))
        c.x.copy_(torch.randn(c.x.shape, device=DEV).to(BF))
        graph.replay()
        ef, eb = c.forward(), c.backward()
        assert all(torch.equal(a, b) for a, b in zip(ef, fo))
        assert all(torch.equal(a[:388], b[:388]) if a.shape[0] == c.A else torch.equal(a, b)
                   for a, b in zip(eb, out))


def test_two_calls_at_once():
    a, b = Case([200, 300], 256, 256, seed=12), Case([10, 0, 600], 512, 128, k=2, seed=13)
    wa, wb = a.backward(), b.backward()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    oa, ob = tuple(torch.zeros_like(t) for t in wa), tuple(torch.zeros_like(t) for t in wb)
    torch.cuda.synchronize()
    a.backward(out=oa, stream=s)
    b.backward(out=ob)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(wa, oa)) and all(torch.equal(x, y) for x, y in zip(wb, ob))


def test_same_as_the_inference_call():
    """The forward's y is moe_expert_ffn's up to the order of fp32 sums."""
    c = Case([40, 0, 300], 256, 256, k=2, seed=14)
    _, y = c.forward()
    y2 = c.new(c.A, c.H)
    ws = torch.empty(moe.moe_expert_ffn_workspace(c.W, c.T, 2), dtype=torch.uint8, device=DEV)
    moe.moe_expert_ffn(c.W, None, c.x, c.T, 2, c.counts, c.offsets, c.sorted_idx, y2, ws)
    d = (y[:c.n].double() - y2[:c.n].double()).norm() / y2[:c.n].double().norm()
    assert float(d) <= 1.5 * math.sqrt(2) * B / math.sqrt(3)


def test_binding_refuses():
    c = Case([8, 8], 128, 128, seed=15)
    gu, y = c.new(16, 256), c.new(16, 128)
    base = dict(x=c.x, counts=c.counts, offsets=c.offsets, sorted_idx=c.sorted_idx, gate_up=gu, rows=y, ws=c.ws)
    for bad in (dict(x=c.x.float()), dict(x=c.x[:15]), dict(counts=c.counts[:1]), dict(offsets=c.offsets[:2]),
                dict(sorted_idx=c.sorted_idx.long()), dict(sorted_idx=c.sorted_idx[:15]), dict(gate_up=gu[:15]),
                dict(rows=y[:, :64]), dict(ws=c.ws.float()), dict(counts=c.counts.cpu())):
        a = base | bad
        args = (c.W, a["x"], 16, 1, a["counts"], a["offsets"], a["sorted_idx"], a["gate_up"], a["rows"], a["ws"])
        with pytest.raises(ValueError):
            moe.moe_expert_ffn_train(*args)
        with pytest.raises(ValueError):
            moe.moe_expert_ffn_backward(*args, d_x_perm=c.new(16, 128))
    args = (c.W, c.x, 16, 1, c.counts, c.offsets, c.sorted_idx, gu, y, c.ws)
    d13, d2 = c.new(2, 256, 128), c.new(2, 128, 128)
    for kw in (dict(d_w13=d13, d_w2=d2.float()), dict(d_w13=d13.half()), dict(d_w13=d13[:1]),
               dict(d_x_perm=y[:15])):
        with pytest.raises(ValueError):
            moe.moe_expert_ffn_backward(*args, **kw)
    with pytest.raises(moe.MoeError) as err:
        moe.moe_expert_ffn_backward(*args, d_w13=d13, accumulate=True)
    assert err.value.status == moe.MOE_ERR_UNSUPPORTED
    with pytest.raises(moe.MoeError) as err:
        moe.moe_expert_ffn_train(*args[:-1], c.ws[:256])
    assert err.value.status == moe.MOE_ERR_WORKSPACE


def test_binding_refuses_rows_of_another_width():
    """Longer buffers are taken, wider rows are not (their rows would be read out of place)."""
    c = Case([8, 8], 128, 128, seed=16)
    wide, gu, y = c.new(16, 256), c.new(16, 256), c.new(16, 128)
    good = [c.W, c.x, 16, 1, c.counts, c.offsets, c.sorted_idx, gu, y, c.ws]
    for at, bad in ((1, wide), (7, c.new(16, 512)), (8, wide)):
        args = good[:at] + [bad] + good[at + 1:]
        with pytest.raises(ValueError):
            moe.moe_expert_ffn_train(*args)
        with pytest.raises(ValueError):
            moe.moe_expert_ffn_backward(*args, d_x_perm=c.new(16, 128))
    with pytest.raises(ValueError):
        moe.moe_expert_ffn_backward(*good, d_x_perm=wide)
    moe.moe_expert_ffn_train(*good[:7], c.new(32 * 256), c.new(20, 128), c.ws)


@pytest.mark.parametrize("gathered", [False, True])
def test_offsets_past_32_bits(gathered):
    """140000 rows of which the last 260 belong to experts: gate_up and its gradient have more than
    2^32 elements."""
    n, H, I, A = [100, 0, 160], 128, 16384, 140000
    flush(f"[train] offsets past 32 bits, gathered={gathered}")
    c = Case(n, H, I, seed=17, gathered=gathered)
    first = A - c.n
    gu, y, dx = c.new(A, 2 * I), c.new(A, H), c.new(A, H)
    d13, d2 = c.new(3, 2 * I, H, dtype=F32), c.new(3, H, I, dtype=F32)
    ws = torch.empty(moe.moe_expert_ffn_backward_workspace(c.W, A, 1), dtype=torch.uint8, device=DEV)
    x, dy = torch.zeros((A, H), dtype=BF, device=DEV), torch.zeros((A, H), dtype=BF, device=DEV)
    x[first:], dy[first:] = c.rows, c.dy
    order = None
    if gathered:  # the rows in use come from the first tokens
        x[:c.n], x[first:] = c.rows, 0
        order = (torch.arange(A, device=DEV) - first).remainder(A).int()
    c.offsets += first
    moe.moe_expert_ffn_train(c.W, x, A, 1, c.counts, c.offsets, order, gu, y, ws)
    torch.cuda.synchronize()
    assert bool((gu[:first:1000] == MARK).all()) and bool((y[:first] == MARK).all())
    check_forward(c, gu[first:], y[first:], A)
    gu[first:] = c.gu
    moe.moe_expert_ffn_backward(c.W, x, A, 1, c.counts, c.offsets, order, gu, dy, ws, dx, d13, d2)
    torch.cuda.synchronize()
    assert bool((dx[:first] == MARK).all())
    check_backward(c, dx[first:], d13, d2, rows=A)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_weights_past_32_bits(dtype):
    """9 experts of 16384 x 16384, rows in the last: the weights and their gradients have more than
    2^32 elements."""
    E, H, I, n = 9, 16384, 16384, 70
    flush(f"[train] weights past 32 bits {dtype}")
    c = Case([n], H, I, seed=18, gathered=False)
    rec = torch.zeros((E, c.rec.shape[1]), dtype=BF, device=DEV)
    rec[E - 1] = c.rec[0]
    W = moe.experts("bf16", E, H, I, rec, rec.shape[1] * 2)
    counts, offsets = torch.zeros(E, dtype=torch.int32, device=DEV), torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    counts[-1], offsets[-1] = n, n
    gu, y, dx = c.new(n, 2 * I), c.new(n, H), c.new(n, H)
    moe.moe_expert_ffn_train(W, c.x, n, 1, counts, offsets, None, gu, y, c.ws)
    torch.cuda.synchronize()
    check_forward(c, gu, y)
    d13, d2 = c.new(E, 2 * I, H, dtype=dtype), c.new(E, H, I, dtype=dtype)
    moe.moe_expert_ffn_backward(W, c.x, n, 1, counts, offsets, None, c.gu, c.dy, c.ws, dx, d13, d2)
    torch.cuda.synchronize()
    check_backward(c, dx, d13[E - 1:], d2[E - 1:])
    assert not bool(d13[:E - 1].any()) and not bool(d2[:E - 1].any())


def test_two_graphs_share_a_workspace():
    """Replayed in turn on one stream, each with other eager calls between."""
    a, b = Case([200, 0, 300], 256, 256, k=2, seed=19), Case([10, 600], 512, 256, seed=20)
    if b.ws.numel() > a.ws.numel():
        a.ws = b.ws
    else:
        b.ws = a.ws
    want = [[t.clone() for t in (*c.forward(), *c.backward())] for c in (a, b)]
    outs, graphs = [], []
    for c in (a, b):
        fo = (c.new(c.A, 2 * c.I), c.new(c.A, c.H))
        bo = (c.new(c.A, c.H), c.new(c.E, 2 * c.I, c.H), c.new(c.E, c.H, c.I))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.moe_expert_ffn_train(c.W, c.x, c.T, c.k, c.counts, c.offsets, c.sorted_idx, *fo, c.ws)
            c.backward(out=bo)
        outs.append((*fo, *bo))
        graphs.append(g)
    for r in range(4):
        for i in ((0, 1), (1, 0), (0, 0), (1, 1))[r]:
            for t in outs[i]:
                t.zero_()
            graphs[i].replay()
            (b, a)[i].backward()
            c = (a, b)[i]
            for got, w in zip(outs[i], want[i]):
                n = c.n if got.shape[0] == c.A else len(got)
                assert torch.equal(got[:n], w[:n])


def test_smaller_batches_in_a_larger_ones_workspace():
    """A workspace for 97 rows holds what any batch of fewer needs (their parts are two)."""
    for E, H, I, k in ((3, 128, 128, 1), (2, 256, 384, 3)):
        W = moe.experts("bf16", E, H, I, torch.empty(E * 3 * H * I, dtype=BF, device=DEV), 6 * H * I)
        for f in (moe.moe_expert_ffn_train_workspace, moe.moe_expert_ffn_backward_workspace):
            sizes = [f(W, T, k) for T in range(1, 300)]
            assert sizes == sorted(sizes)


@pytest.mark.parametrize("n", [9, 200])
def test_infinities_stay_infinite(n):
    """An infinite weight or row against values that bf16 holds exactly (whose second part is nothing)
    and ones that it does not: infinite results, not NaN."""
    H = I = 128
    c = Case([n], H, I, gathered=False, seed=21)
    c.gu[:] = torch.randn(n, 2 * I, device=DEV).to(BF)
    c.gu[:, :I] = 300.0                 # silu(g) = g: h = 300 u, exact and not
    c.gu[0, I:] = 2.0
    c.dy.abs_()
    rec = c.rec.clone()
    w13, w2 = rec[0, :2 * I * H].view(2 * I, H), rec[0, 2 * I * H:].view(H, I)
    w2[:] = 0.25
    w13[I:] = 0.0
    w13[I + 5, 7] = float("inf")        # dx[:, 7] = du[:, 5] inf + finite ones, du > 0
    W = moe.experts("bf16", 1, H, I, rec, rec.shape[1] * 2)
    dx, d13, d2 = c.new(n, H), c.new(1, 2 * I, H), c.new(1, H, I)
    c.gu[:, I:].abs_()
    c.gu[:, I + 9] = float("inf")       # h[:, 9] = inf: d_w2[:, 9]
    moe.moe_expert_ffn_backward(W, c.x, n, 1, c.counts, c.offsets, None, c.gu, c.dy, c.ws, dx, d13, d2)
    assert bool((d2[0, :, 9] == float("inf")).all())
    assert not bool(d2[0, :, :9].isinf().any()) and not bool(d2[0, :, :9].isnan().any())
    c.gu[:, I + 9] = 1.0
    moe.moe_expert_ffn_backward(W, c.x, n, 1, c.counts, c.offsets, None, c.gu, c.dy, c.ws, dx, d13, d2)
    assert bool((dx[:, 7] == float("inf")).all())
    assert bool(dx[:, :7].isfinite().all()) and bool(dx[:, 8:].isfinite().all())
