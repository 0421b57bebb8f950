"""moe_dispatch, moe_dispatch_backward and moe_combine_backward on the GPU against the float64
oracle.

Tolerances.  eps = 2^-24 (fp32), b = 2^-8 (half a step of bf16).  A scattered row is one fp32
product rounded once more: bit-equal to the same two roundings in torch (a copy without
weights).  A gathered sum adds k products and one addend in fp32: off by (k + 1) eps times the
sum of the magnitudes, then b of the result.  A dot of H products is off by at most H eps
times the sum of its products' magnitudes.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_cases import flush
from oracle import train as OT

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_expert_ffn_router_amd as moe  # noqa: E402

DEV = torch.device("cuda")
EPS, B = 2.0 ** -24, 2.0 ** -8
BF = torch.bfloat16
MARK = 3.5


class Rows:
    """A batch: tokens, a permutation of its assignments, of which `drop` have no row; R rows."""

    def __init__(self, T, k, H, seed=0, drop=0, spare=0):
        g = torch.Generator().manual_seed(seed)
        self.T, self.k, self.H = T, k, H
        A = T * k
        self.R = A + spare
        inv = torch.randperm(self.R, generator=g)[:A].int()
        lost = torch.randperm(A, generator=g)[:drop]
        inv[lost] = torch.tensor([-1, self.R, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32).repeat(drop)[:drop]
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.h = dict(inv=inv, w=torch.softmax(rnd(T, k), 1), x=rnd(T, H).to(BF), add=rnd(T, H).to(BF),
                      rows=rnd(self.R, H).to(BF))
        self.d = {n: t.to(DEV) for n, t in self.h.items()}

    def f64(self, name):
        t = self.h[name]
        return t.double().numpy() if t.is_floating_point() else t.numpy()


# k covers every register count; H: one lane, less than, just and more than one wave's and one
# workgroup's columns, on both sides of the split over a workgroup's waves
CASES = [(1, 1, 8, 0, 0), (1, 16, 2048, 0, 0), (3, 2, 40, 2, 5), (64, 2, 256, 0, 0), (333, 4, 2048, 9, 0),
         (17, 3, 520, 4, 1), (9, 9, 4104, 11, 2), (40, 8, 7168, 0, 0), (4099, 2, 512, 20, 3),
         (4097, 5, 72, 0, 0), (4200, 8, 1032, 31, 0), (5000, 16, 24, 7, 7)]


@pytest.mark.parametrize("T,k,H,drop,spare", CASES)
def test_scatter(T, k, H, drop, spare):
    flush(f"[rows] scatter T={T} k={k} H={H}")
    c = Rows(T, k, H, seed=T + H, drop=drop, spare=spare)
    d = c.d
    ok = (d["inv"] >= 0) & (d["inv"] < c.R)
    tok = torch.arange(T * k, device=DEV)[ok] // k
    at = d["inv"][ok].long()
    for w in (None, d["w"]):
        want = torch.full((c.R, H), MARK, dtype=BF, device=DEV)
        rows = d["x"][tok]
        want[at] = rows if w is None else (rows.float() * w.reshape(-1)[ok][:, None]).to(BF)
        got = torch.full((c.R, H), MARK, dtype=BF, device=DEV)
        moe.moe_dispatch(d["x"], d["inv"], k, got, topk_w=w)
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    # the combine's gradient: the weighted rows, and the dots
    got = torch.full((c.R, H), MARK, dtype=BF, device=DEV)
    dw = torch.full((T, k), MARK, device=DEV)
    moe.moe_combine_backward(d["x"], d["inv"], d["w"], k, got, y_perm=d["rows"], d_topk_w=dw)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    _, exact = OT.combine_backward(c.f64("x"), c.f64("rows"), c.f64("inv"), c.f64("w"))
    _, size = OT.combine_backward(np.abs(c.f64("x")), np.abs(c.f64("rows")), c.f64("inv"), c.f64("w"))
    assert (np.abs(dw.cpu().numpy() - exact) <= H * EPS * size).all()
    # without the dots; and in place of y_perm
    again = torch.full((c.R, H), MARK, dtype=BF, device=DEV)
    moe.moe_combine_backward(d["x"], d["inv"], d["w"], k, again)
    assert torch.equal(again, got)
    own, dw2 = d["rows"].clone(), torch.empty_like(dw)
    moe.moe_combine_backward(d["x"], d["inv"], d["w"], k, own, y_perm=own, d_topk_w=dw2)
    assert torch.equal(own[at], got[at]) and torch.equal(dw2, dw)
    free = torch.ones(c.R, dtype=torch.bool, device=DEV)
    free[at] = False
    assert torch.equal(own[free], d["rows"][free])


@pytest.mark.parametrize("T,k,H,drop,spare", CASES)
@pytest.mark.parametrize("weighted", [False, True])
def test_gather(T, k, H, drop, spare, weighted):
    flush(f"[rows] gather T={T} k={k} H={H} weighted={weighted}")
    c = Rows(T, k, H, seed=T + H + 1, drop=drop, spare=spare)
    d = c.d
    w = d["w"] if weighted else None
    w64 = c.f64("w") if weighted else None
    args = (c.f64("rows"), c.f64("inv"), w64, c.f64("x"))
    size = tuple(np.abs(a) if isinstance(a, np.ndarray) and a.dtype == np.float64 else a for a in args)
    for add in (None, "add"):
        exact, dots = OT.dispatch_backward(*args, None if add is None else c.f64(add))
        mag, dmag = OT.dispatch_backward(*size, None if add is None else np.abs(c.f64(add)))
        out = torch.full((T, H), MARK, dtype=BF, device=DEV)
        dw = torch.full((T, k), MARK, device=DEV)
        moe.moe_dispatch_backward(d["rows"], d["inv"], k, out, topk_w=w, d_add=None if add is None else
                                  d[add], x=d["x"], d_topk_w=dw)
        err = np.abs(out.double().cpu().numpy() - exact)
        assert (err <= (k + 2) * EPS * mag + B * np.abs(exact)).all()
        assert (np.abs(dw.cpu().numpy() - dots) <= H * EPS * dmag).all()
        plain = torch.full((T, H), MARK, dtype=BF, device=DEV)
        moe.moe_dispatch_backward(d["rows"], d["inv"], k, plain, topk_w=w,
                                  d_add=None if add is None else d[add])
        assert torch.equal(plain, out)
    # d_x in place of d_add
    own = d["add"].clone()
    moe.moe_dispatch_backward(d["rows"], d["inv"], k, own, topk_w=w, d_add=own)
    assert torch.equal(own, out)


@pytest.mark.parametrize("k,H,T", [(8, 4096, 4300), (2, 16384, 4300), (16, 2048, 4300), (4, 1032, 33000),
                                   (8, 512, 33000), (4, 256, 132000), (2, 504, 134000), (16, 136, 62000)])
def test_rows_of_more_than_the_caches_hold(k, H, T):
    """Batches that pass the caches by: the same results as in two halves, which do not (each token's
    are its own), and as in 64 bits."""
    flush(f"[rows] large k={k} H={H} T={T}")
    g = torch.Generator(device=DEV).manual_seed(k)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    A = T * k
    x, rows, w = rnd(T, H).to(BF), rnd(A, H).to(BF), torch.softmax(rnd(T, k), 1).contiguous()
    inv = torch.randperm(A, generator=g, device=DEV).int()
    inv[7] = -1
    out, dy = torch.full((A, H), MARK, dtype=BF, device=DEV), torch.full((A, H), MARK, dtype=BF, device=DEV)
    dx, dw, dw2 = torch.empty_like(x), torch.empty(T, k, device=DEV), torch.empty(T, k, device=DEV)
    moe.moe_dispatch(x, inv, k, out, topk_w=w)
    moe.moe_combine_backward(x, inv, w, k, dy, y_perm=rows, d_topk_w=dw)
    moe.moe_dispatch_backward(rows, inv, k, dx, topk_w=w, d_add=x, x=x, d_topk_w=dw2)
    assert torch.equal(out, dy)
    ok = inv >= 0
    at, tok = inv[ok].long(), (torch.arange(A, device=DEV) // k)[ok]
    assert torch.equal(out[at], (x[tok].float() * w.reshape(-1)[ok][:, None]).to(BF))
    assert int((out == MARK).all(1).sum()) == 1
    h = T // 2
    for part in (slice(0, h), slice(h, T)):
        i, p = inv[part.start * k:part.stop * k].contiguous(), x[part].contiguous()
        o, d = torch.empty_like(p), torch.empty(p.shape[0], k, device=DEV)
        moe.moe_dispatch_backward(rows, i, k, o, topk_w=w[part].contiguous(), d_add=p, x=p, d_topk_w=d)
        assert torch.equal(o, dx[part])   # (the dots' order of columns is another there)
    r64 = torch.where(ok.view(T, k, 1), rows[inv.clamp(min=0).long()].view(T, k, H).double(), 0.0)
    dots, size = (r64 * x.double()[:, None]).sum(2), (r64.abs() * x.double().abs()[:, None]).sum(2)
    for d in (dw, dw2):
        assert bool(((d.double() - dots).abs() <= H * EPS * size).all())
    want = (r64 * w.double()[:, :, None]).sum(1) + x.double()
    mag = (r64.abs() * w.double()[:, :, None]).sum(1) + x.double().abs()
    assert bool(((dx.double() - want).abs() <= (k + 2) * EPS * mag + B * want.abs()).all())


def test_all_dropped_and_no_rows():
    T, k, H = 5, 3, 64
    x = torch.randn(T, H, device=DEV).to(BF)
    inv = torch.full((T * k,), -1, dtype=torch.int32, device=DEV)
    none = torch.empty(0, H, dtype=BF, device=DEV)
    out, dw = torch.full((T, H), MARK, dtype=BF, device=DEV), torch.full((T, k), MARK, device=DEV)
    moe.moe_dispatch(x, inv, k, none)
    moe.moe_dispatch_backward(none, inv, k, out, d_add=x, x=x, d_topk_w=dw)
    assert torch.equal(out, x) and not dw.any()
    dw.fill_(MARK)
    moe.moe_combine_backward(x, inv, torch.rand(T, k, device=DEV), k, none, y_perm=none, d_topk_w=dw)
    assert not dw.any()


def test_no_tokens():
    x = torch.empty(0, 64, dtype=BF, device=DEV)
    inv, w = torch.empty(0, dtype=torch.int32, device=DEV), torch.empty(0, 2, device=DEV)
    rows = torch.full((4, 64), MARK, dtype=BF, device=DEV)
    # no tokens: every tensor of theirs is empty, and so is its device pointer
    with pytest.raises(ValueError):
        moe.moe_dispatch(torch.empty(0, 64, dtype=BF), inv, 2, rows)
    moe.moe_dispatch(x, inv, 2, rows, topk_w=w)
    moe.moe_dispatch_backward(rows, inv, 2, x, topk_w=w)
    moe.moe_combine_backward(x, inv, w, 2, rows, y_perm=rows, d_topk_w=w)
    assert bool((rows == MARK).all())


def test_values_that_are_not_finite():
    """A copy keeps every bit; products and sums follow the formulas; other rows are untouched by them."""
    T, k, H = 6, 2, 128
    c = Rows(T, k, H, seed=5)
    x = c.d["x"].clone()
    x.view(torch.int16)[0, :4] = torch.tensor([0x7f81, -1, 0x7f80, -0x80], dtype=torch.int16, device=DEV)
    inv = c.d["inv"].long()
    got = torch.empty(c.R, H, dtype=BF, device=DEV)
    moe.moe_dispatch(x, c.d["inv"], k, got)
    assert torch.equal(got[inv[0]].view(torch.int16), x[0].view(torch.int16))
    moe.moe_dispatch(x, c.d["inv"], k, got, topk_w=c.d["w"])
    want = (x[torch.arange(T * k, device=DEV) // k].float() * c.d["w"].reshape(-1)[:, None]).to(BF)
    assert torch.equal(torch.nan_to_num(got[inv], nan=7.0), torch.nan_to_num(want, nan=7.0))
    rows = c.d["rows"].clone()
    rows[inv[3]] = float("nan")
    out, dw = torch.empty(T, H, dtype=BF, device=DEV), torch.empty(T, k, device=DEV)
    moe.moe_dispatch_backward(rows, c.d["inv"], k, out, x=c.d["x"], d_topk_w=dw)
    assert bool(out[1].isnan().all()) and not bool(out[[0, 2, 3, 4, 5]].isnan().any())
    assert dw.isnan().nonzero().tolist() == [[1, 1]]


def test_offsets_past_32_bits():
    """Rows whose elements lie past 2^32: the last ones of a 9 GB buffer."""
    H, k, T = 16384, 2, 3
    R = (1 << 32) // H + 64
    big = torch.empty(R, H, dtype=BF, device=DEV)
    big[-64:] = MARK
    x = torch.randn(T, H, device=DEV).to(BF)
    inv = torch.tensor([R - 1, R - 5, R - 9, 3, R - 30, R - 2], dtype=torch.int32, device=DEV)
    flush("[rows] past 32 bits")
    moe.moe_dispatch(x, inv, k, big)
    assert torch.equal(big[inv.long()], x.repeat_interleave(k, 0))
    assert bool((big[R - 4:R - 2] == MARK).all())
    out = torch.empty_like(x)
    moe.moe_dispatch_backward(big, inv, k, out)
    assert torch.equal(out, (x.float() * 2).to(BF))


def test_other_stream_and_graph():
    T, k, H = 333, 4, 512
    c = Rows(T, k, H, seed=9)
    d = c.d
    want = torch.empty(c.R, H, dtype=BF, device=DEV)
    moe.moe_dispatch(d["x"], d["inv"], k, want, topk_w=d["w"])
    s = torch.cuda.Stream()
    got, out = torch.zeros_like(want), torch.zeros(T, H, dtype=BF, device=DEV)
    dw = torch.zeros(T, k, device=DEV)
    s.wait_stream(torch.cuda.current_stream())
    moe.moe_dispatch(d["x"], d["inv"], k, got, topk_w=d["w"], stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_dispatch(d["x"], d["inv"], k, got, topk_w=d["w"])
        moe.moe_dispatch_backward(got, d["inv"], k, out, topk_w=d["w"], x=d["x"], d_topk_w=dw)
    for r in range(3):
        d["x"].copy_(torch.randn(T, H, device=DEV).to(BF))
        g.replay()
        e_rows, e_out, e_dw = torch.empty_like(got), torch.empty_like(out), torch.empty_like(dw)
        moe.moe_dispatch(d["x"], d["inv"], k, e_rows, topk_w=d["w"])
        moe.moe_dispatch_backward(e_rows, d["inv"], k, e_out, topk_w=d["w"], x=d["x"], d_topk_w=e_dw)
        assert torch.equal(got, e_rows) and torch.equal(out, e_out) and torch.equal(dw, e_dw)


def test_binding_refuses():
    c = Rows(4, 2, 64)
    d = c.d
    out = torch.empty(c.R, 64, dtype=BF, device=DEV)
    for bad in (dict(x=d["x"].float()), dict(inv=d["inv"].long()), dict(inv=d["inv"][:-1]),
                dict(out=out[:, :32]), dict(w=d["w"].double()), dict(w=d["w"][:-1]), dict(x=d["x"].cpu()),
                dict(x=d["x"].t()), dict(inv=d["inv"].cpu())):
        a = dict(x=d["x"], inv=d["inv"], out=out, w=d["w"]) | bad
        with pytest.raises(ValueError):
            moe.moe_dispatch(a["x"], a["inv"], 2, a["out"], topk_w=a["w"])
    with pytest.raises(moe.MoeError):
        moe.moe_dispatch_backward(out, d["inv"], 2, d["x"], d_topk_w=d["w"])   # no x
    with pytest.raises(moe.MoeError):
        moe.moe_dispatch(d["x"][:, :60].contiguous(), d["inv"], 2, out[:, :60].contiguous())
