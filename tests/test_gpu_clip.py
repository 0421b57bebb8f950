"""moe_clip_grad_norm on the GPU.

Tolerances.  The sums are in 64 bits, so the norm is one fp32 rounding (2^-24) off plus the
64-bit sum's n 2^-53: 2^-23 covers it.  The scale is one division in 64 bits and one rounding
to fp32 (2^-24); a clipped fp32 element one more (2^-22 in all), a bf16 one half a step of bf16
(2^-8) and its fp32 product's 2^-23.  Subnormal results: half of the smallest step besides.
"""
from __future__ import annotations

import math

import pytest
import torch

from gpu_cases import flush

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_expert_ffn_router_amd as moe  # noqa: E402

DEV = torch.device("cuda")
BF, F32 = torch.bfloat16, torch.float32
MARK = 3.5


def make(sizes, seed=0, offsets=True):
    """Gradients (alternating types) as views at odd element offsets of larger buffers."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    ts, bufs = [], []
    for i, n in enumerate(sizes):
        off = (i * 3) % 11 if offsets else 0
        buf = torch.full((n + off + 9,), MARK, dtype=F32 if i % 2 else BF, device=DEV)
        buf[off:off + n] = (torch.randn(n, generator=g, device=DEV) * 10.0 ** (i % 4 - 2)).to(buf.dtype)
        ts.append(buf[off:off + n])
        bufs.append((buf, off))
    return ts, bufs


def call(grads, max_norm, clipped=None, ws=None, stream=None):
    ns = torch.full((2,), -1.0, device=DEV)
    if ws is None:
        ws = torch.full((moe.moe_clip_grad_norm_workspace(len(grads)),), 0xff, dtype=torch.uint8,
                        device=DEV)
    moe.moe_clip_grad_norm(grads, max_norm, ns, ws, clipped=clipped, stream=stream)
    return ns


def check(ns, grads, max_norm, clipped):
    norm = math.sqrt(sum(float(t.double().square().sum()) for t in grads))
    scale = min(1.0, max_norm / (norm + 1e-6))
    got = ns.tolist()
    assert abs(got[0] - norm) <= 2.0 ** -23 * norm
    assert abs(got[1] - scale) <= 2.0 ** -22 * scale
    for t, c in zip(grads, clipped or []):
        want = t.double() * scale
        tol = (2.0 ** -22 if t.dtype is F32 else 2.0 ** -8 + 2.0 ** -22) * want.abs() + 2.0 ** -133
        assert bool(((c.double() - want).abs() <= tol).all())


SIZES = [[1], [7], [8], [16383], [16384], [16385, 1, 0, 5], [40000, 8191, 33], [3] * 128, [5, 0] * 70,
         [1000 + i for i in range(300)], [1 << 22, 3, (1 << 20) + 1, 12345], [0], []]


@pytest.mark.parametrize("i", range(len(SIZES)))
@pytest.mark.parametrize("max_norm", [0.01, 1e9])
def test_clip(i, max_norm):
    flush(f"[clip] sizes {SIZES[i][:5]} max_norm {max_norm}")
    grads, bufs = make(SIZES[i], seed=i)
    outs, obufs = make(SIZES[i], seed=100 + i, offsets=i % 2 == 0)   # aligned alike, or not
    keep = [t.clone() for t in grads]
    ns = call(grads, max_norm, outs)
    check(ns, keep, max_norm, outs)
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    for (b, off), t in zip(obufs, outs):   # nothing beside them
        assert bool((b[:off] == MARK).all()) and bool((b[off + t.numel():] == MARK).all())
    assert torch.equal(call(grads, max_norm), ns)
    # in place
    assert torch.equal(call(grads, max_norm, grads), ns)
    assert all(torch.equal(a, b) for a, b in zip(grads, outs))
    for (b, off), t in zip(bufs, grads):
        assert bool((b[:off] == MARK).all()) and bool((b[off + t.numel():] == MARK).all())


def test_no_clipping_changes_nothing():
    grads, _ = make([1000, 1001], seed=3)
    keep = [t.clone() for t in grads]
    ns = call(grads, float("inf"), grads)
    assert ns[1] == 1 and all(torch.equal(a, b) for a, b in zip(grads, keep))
    outs = [torch.empty_like(t) for t in grads]
    call(grads, float("inf"), outs)
    assert all(torch.equal(a, b) for a, b in zip(outs, keep))
    assert call(grads, 0.0, outs)[1] == 0 and not any(o.any() for o in outs)


def test_extreme_values():
    """Squares past fp32's range on both sides."""
    for v in (1e30, 1e-30):
        t = torch.full((4096,), v, device=DEV)
        ns = call([t], 1.0, [t])
        assert float(ns[0]) == pytest.approx(64 * v, rel=1e-6)
    ns = call([torch.full((16,), 2.0 ** 100, dtype=BF, device=DEV), torch.ones(3, device=DEV)], 1.0)
    assert float(ns[0]) == pytest.approx(4 * 2.0 ** 100, rel=1e-6)


def test_values_that_are_not_finite():
    t = torch.ones(5000, device=DEV)
    t[4321] = float("inf")
    u = torch.full((100,), 2.0, dtype=BF, device=DEV)
    ns = call([t, u], 1.0, [t, u])
    assert ns.tolist() == [math.inf, 0.0]
    assert not u.any() and int(t.isnan().sum()) == 1 and bool(t[4321].isnan())
    t = torch.ones(5000, device=DEV)
    t[17] = float("nan")
    ns = call([t, u], 1.0)
    assert bool(ns.isnan().all())


def test_no_limit():
    """max_norm infinity: the scale is 1 whatever the norm, NaN for a NaN norm alone."""
    t = torch.arange(1.0, 6000.0, device=DEV)
    u = torch.full((100,), 2.0, dtype=BF, device=DEV)
    assert float(call([t, u], math.inf, [t, u])[1]) == 1.0
    t[77] = -float("inf")
    keep, out = t.clone(), [torch.zeros_like(t), torch.zeros_like(u)]
    ns = call([t, u], math.inf, out)
    assert ns.tolist() == [math.inf, 1.0]
    assert torch.equal(out[0], keep) and torch.equal(out[1], u)
    t[78] = float("nan")
    assert bool(call([t, u] * 70, math.inf).isnan().all())


def test_many_elements():
    """A tensor of more than 2^31 bytes, and one element past 2^31 in a bf16 one."""
    flush("[clip] 2^31 + 5 elements")
    n = (1 << 31) + 5
    t = torch.zeros(n, dtype=BF, device=DEV)
    t[-1], t[0], t[1 << 30] = 3.0, 4.0, 12.0
    ns = call([t], 1.3, [t])
    assert float(ns[0]) == pytest.approx(13.0, rel=1e-6)
    assert float(t[-1]) == pytest.approx(0.3, rel=2 ** -7) and float(t[0]) == pytest.approx(0.4, rel=2 ** -7)


def test_more_than_the_caches_hold():
    """Passes that bypass the caches, into other tensors aligned alike and not."""
    flush("[clip] 500 MB")
    grads, _ = make([1 << 27, 60_000_001, 77], seed=8)
    outs, obufs = make([1 << 27, 60_000_001, 77], seed=9)
    ns = call(grads, 2.0, outs)
    check(ns, grads, 2.0, outs)
    outs2, _ = make([1 << 27, 60_000_001, 77], seed=9, offsets=False)
    assert torch.equal(call(grads, 2.0, outs2), ns)
    assert all(torch.equal(a, b) for a, b in zip(outs, outs2))
    for (b, off), t in zip(obufs, outs):
        assert bool((b[:off] == MARK).all()) and bool((b[off + t.numel():] == MARK).all())


def test_repeated_calls_and_streams_and_graph():
    grads, _ = make([70000, 4097, 13], seed=4)
    outs = [torch.empty_like(t) for t in grads]
    ns = call(grads, 0.5, outs)
    for _ in range(3):
        again = [torch.empty_like(t) for t in grads]
        assert torch.equal(call(grads, 0.5, again), ns)
        assert all(torch.equal(a, b) for a, b in zip(outs, again))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other, _ = make([70000, 4097, 13], seed=5)
    torch.cuda.synchronize()
    ws = [torch.empty(moe.moe_clip_grad_norm_workspace(3), dtype=torch.uint8, device=DEV) for _ in range(2)]
    out2 = [torch.empty_like(t) for t in grads]
    n2, n1 = torch.empty(2, device=DEV), torch.empty(2, device=DEV)
    torch.cuda.synchronize()
    moe.moe_clip_grad_norm(other, 0.5, n2, ws[0], clipped=out2, stream=s)   # two calls at once
    moe.moe_clip_grad_norm(grads, 0.5, n1, ws[1], clipped=outs)
    torch.cuda.synchronize()
    assert torch.equal(n1, ns)
    check(n2, other, 0.5, out2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_clip_grad_norm(grads, 0.5, n1, ws[1], clipped=outs)
    for r in range(3):
        for t in grads:
            t.mul_(1.5)
        g.replay()
        check(n1, grads, 0.5, outs)


def test_binding_refuses():
    a, b = torch.ones(8, device=DEV), torch.ones(8, dtype=BF, device=DEV)
    ns = torch.empty(2, device=DEV)
    ws = torch.empty(moe.moe_clip_grad_norm_workspace(2), dtype=torch.uint8, device=DEV)
    for grads, clipped in (([a.half()], None), ([a.cpu()], None), ([torch.ones(8, 8, device=DEV).t()], None),
                           ([a, b], [a]), ([a], [b]), ([a], [a[:4]]), ([a], [torch.ones(8)])):
        with pytest.raises(ValueError):
            moe.moe_clip_grad_norm(grads, 1.0, ns, ws, clipped=clipped)
    for grads, clipped in (([a, a], [a, a]), ([a[:4], a[2:6]], [a[:4], a[2:6]])):
        with pytest.raises(moe.MoeError):
            moe.moe_clip_grad_norm(grads, 1.0, ns, ws, clipped=clipped)
    assert float(call([a, a], 1.0)[0]) == 4.0    # twice the same, only measured
