"""What the expert training calls promise, on the kernels of every tile size: accumulation, outputs left out,
whole numbers bit by bit, values that are not finite, repetition, streams, graphs whose batch changes, two
calls at once.  (Accuracy over sizes and the same promises on small layers: test_gpu_expert_train.)  Every
size names the sides of the tiles it takes, so that each product meets 64, 128 and 256.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_cases import flush
from train_tiles import sides

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_expert_ffn_router_amd as moe  # noqa: E402
from test_gpu_expert_train import BF, DEV, F32, MARK, Case, check_backward  # noqa: E402

# experts without rows first, last and between, segments in whole blocks of 64 and not, rows behind the last;
# sides of gate_up, down, dh, dx, w13, w2
SIZES = {
    "small": (dict(counts=[0, 70, 0, 64, 1, 129, 0], H=384, I=256, k=2, behind=3), (64, 64, 64, 64, 64, 64)),
    "mixed": (dict(counts=[0, 180, 192, 257, 0, 64, 1, 300, 250, 129, 320, 333, 0], H=1024, I=640, k=2, behind=6),
              (64, 64, 64, 64, 256, 128)),
    "middling": (dict(counts=[0, 1000, 1300, 513, 1100, 1023, 0], H=1024, I=512, k=3, behind=5),
                 (128, 128, 64, 128, 128, 64)),
    "large": (dict(counts=[0, 600, 1024, 257, 0, 1, 999, 64, 1000, 333, 0], H=2048, I=1024, k=2, behind=7),
              (256, 256, 128, 256, 256, 256)),
    "wide": (dict(counts=[0, 1100, 1345, 0, 960, 995], H=1024, I=2048, k=1, gathered=False, behind=4),
             (256, 64, 256, 64, 256, 128)),
}
PRODUCTS = ("gate_up", "down", "dh", "dx", "w13", "w2")


def case(name, seed, **over):
    spec, want = SIZES[name]
    c = Case(**(spec | over), seed=seed)
    assert tuple(sides(c.E, c.H, c.I, c.A)[p] for p in PRODUCTS) == want
    return c


def same(a, b, n, A):
    """Equal bits in the rows in use (of A) or everywhere, NaN in no place."""
    return all(torch.equal(x[:n], y[:n]) if x.shape[0] == A else torch.equal(x, y) for x, y in zip(a, b))


def test_every_kernel_is_met():
    met = {(p, s) for _, want in SIZES.values() for p, s in zip(PRODUCTS, want)}
    assert met == {(p, s) for p in PRODUCTS for s in (64, 128, 256)}


@pytest.mark.parametrize("name", SIZES)
def test_accumulate(name):
    flush(f"[train tiles] accumulate {name}")
    c = case(name, 40)
    full = lambda *s: torch.full(s, 0.25, device=DEV)  # noqa: E731
    out = (c.new(c.A, c.H), full(c.E, 2 * c.I, c.H), full(c.E, c.H, c.I))
    c.backward(accumulate=True, out=out)
    check_backward(c, *out, base=0.25)
    alone = c.backward(F32)
    twice = (out[0], *(t.clone() for t in alone[1:]))
    c.backward(accumulate=True, out=twice)
    for a, t in zip(alone[1:], twice[1:]):
        assert torch.equal(2 * a, t)
    marked = (out[0], c.new(c.E, 2 * c.I, c.H, dtype=F32), c.new(c.E, c.H, c.I, dtype=F32))
    c.backward(accumulate=True, out=marked)
    empty = c.counts == 0
    assert bool(empty.any()) and all(bool((t[empty] == MARK).all()) for t in marked[1:])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("name", SIZES)
def test_outputs_left_out(name, dtype):
    """Each output alone and each left out: large and small tiles of the others in any mixture."""
    flush(f"[train tiles] outputs left out {name} {dtype}")
    c = case(name, 41)
    whole = c.backward(dtype)
    for given in ((0,), (1,), (2,), (0, 1), (0, 2), (1, 2)):
        out = tuple(torch.full_like(t, MARK) if i in given else None for i, t in enumerate(whole))
        c.backward(dtype, out=out)
        assert all(torch.equal(out[i], whole[i]) for i in given), given


@pytest.mark.parametrize("name", SIZES)
def test_whole_numbers_are_exact(name):
    """Sums of small whole numbers lose nothing: gate_up and all three gradients, every product and place."""
    flush(f"[train tiles] whole numbers {name}")
    c = case(name, 42)
    g = torch.Generator(device=DEV).manual_seed(43)
    E, H, I = c.E, c.H, c.I
    ints = lambda t, lo, hi: t.copy_(torch.randint(lo, hi, t.shape, generator=g, device=DEV))  # noqa: E731
    ints(c.x, -2, 3)
    c.rows = c.x[c.sorted_idx.long() // c.k] if c.sorted_idx is not None else c.x
    rec = torch.randint(-1, 2, c.rec.shape, generator=g, device=DEV).to(BF)
    # sparse enough that what is kept as bf16 stays within its 8 bits: 16 terms a sum or so
    rec *= torch.rand(c.rec.shape, generator=g, device=DEV) < 24.0 / max(H, I)
    c.rec.copy_(rec)
    w13, w2 = (t.double() for t in (c.rec[:, :2 * I * H].view(E, 2 * I, H), c.rec[:, 2 * I * H:].view(E, H, I)))
    gu, _ = c.forward()
    # gates of 64 have a sigmoid of 1 and a slope of 1: h = 64 u, du = 64 dh, dg = dh u
    c.gu[:, :I] = 64.0
    c.gu[:, I:] = torch.randint(-2, 3, (c.A, I), generator=g, device=DEV).to(BF)
    ints(c.dy, -1, 2)
    dx, d13, d2 = c.backward(F32)
    for e in range(E):
        p = slice(c.ends[e], c.ends[e + 1])
        x, dy, u = c.rows[p].double(), c.dy[p].double(), c.gu[p, I:].double()
        want = x @ w13[e].t()
        assert bool((want.abs() <= 256).all()) and torch.equal(gu[p].double(), want)
        dh = dy @ w2[e]
        dz = torch.cat([dh * u, 64 * dh], 1)
        assert bool((dh.abs() <= 128).all())
        assert torch.equal(dx[p], (dz @ w13[e]).to(BF))
        assert torch.equal(d13[e].double(), dz.t() @ x)
        assert torch.equal(d2[e].double(), dy.t() @ (64 * u))


@pytest.mark.parametrize("name", SIZES)
def test_values_that_are_not_finite(name):
    """NaN and infinite rows behind the last segment, or of another expert, reach no result."""
    flush(f"[train tiles] not finite {name}")
    c = case(name, 44, k=1)
    n, A = c.n, c.A
    first = (*c.backward(F32), *c.forward())
    bad = c.sorted_idx[n:].long() if c.sorted_idx is not None else torch.arange(n, A, device=DEV)
    c.x[bad], c.gu[n:], c.dy[n:] = float("nan"), float("inf"), float("nan")
    assert same(first, (*c.backward(F32), *c.forward()), n, A)
    e = int(c.counts[:4].argmax())               # the last row of an expert: NaN
    row = int(c.ends[e + 1]) - 1
    c.dy[row] = float("nan")
    dx, d13, d2 = c.backward(F32)
    others = torch.arange(c.E, device=DEV) != e
    assert bool(dx[row].isnan().all()) and torch.equal(dx[:row], first[0][:row])
    assert torch.equal(dx[row + 1:n], first[0][row + 1:n])
    assert bool(d2[e].isnan().all()) and torch.equal(d2[others], first[2][others])
    assert bool(d13[e].isnan().any()) and torch.equal(d13[others], first[1][others])


@pytest.mark.parametrize("name", SIZES)
def test_repeats_and_streams(name):
    flush(f"[train tiles] repeats {name}")
    c = case(name, 45)
    first = (*c.forward(), *c.backward())
    for dtype in (BF, F32):
        base = c.backward(dtype)
        for _ in range(6):
            c.ws.fill_(255)
            assert same(first[:2], c.forward(), c.n, c.A)
            c.ws.fill_(255)
            assert same(base, c.backward(dtype), c.n, c.A)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        got = (*c.forward(stream=s), *c.backward(stream=s))
    s.synchronize()
    assert same(first, got, c.n, c.A)


@pytest.mark.parametrize("name", SIZES)
def test_graph_of_changing_batches(name):
    """Captured once, replayed over other rows and other numbers of rows: none, all in one expert, alike."""
    flush(f"[train tiles] graph {name}")
    c = case(name, 46)
    E, n = c.E, c.n
    out, fo = c.backward(), (c.new(c.A, 2 * c.I), c.new(c.A, c.H))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_expert_ffn_train(c.W, c.x, c.T, c.k, c.counts, c.offsets, c.sorted_idx, *fo, c.ws)
        c.backward(out=out)
    one, alike = [0] * E, [n // E] * E
    one[E - 2] = n
    own = c.counts.tolist()
    for counts in (own, one, [0] * E, alike, own[::-1], own):
        used = sum(counts)
        c.counts.copy_(torch.tensor(counts, dtype=torch.int32))
        c.offsets.copy_(torch.tensor([0] + np.cumsum(counts).tolist(), dtype=torch.int32))
        c.x.copy_(torch.randn(c.x.shape, device=DEV).to(BF))
        for t in (*fo, *out):
            t.fill_(MARK)
        graph.replay()
        eager = (*c.forward(), *c.backward())
        torch.cuda.synchronize()
        for a, b in zip(eager, (*fo, *out)):
            assert torch.equal(a, b), counts
            if a.shape[0] == c.A:
                assert bool((a[used:] == MARK).all())
        if not used:
            assert not bool(eager[3].any()) and not bool(eager[4].any())


def test_two_calls_at_once():
    a, b = case("large", 47), case("mixed", 48)
    want = [(*c.forward(), *c.backward(F32)) for c in (a, b)]
    s = torch.cuda.Stream()
    outs = [tuple(torch.zeros_like(t) for t in w) for w in want]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, o, stream in ((a, outs[0], s), (b, outs[1], None)):
            moe.moe_expert_ffn_train(c.W, c.x, c.T, c.k, c.counts, c.offsets, c.sorted_idx, *o[:2], c.ws, stream=stream)
            c.backward(out=o[2:], stream=stream)
    torch.cuda.synchronize()
    for c, w, o in zip((a, b), want, outs):
        assert same(w, o, c.n, c.A)
