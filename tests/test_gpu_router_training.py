"""moe_balance_loss and moe_route_backward against the float64 oracle on the GPU.

Tolerances.  eps = 2^-24.  With d the distance of a logit from its row's
maximum, exp(x - m) is off by at most (d + 2) eps relative (one rounding of the
difference, one ulp of expf), the row's sum by the probability-weighted mean
of that (at most ln E + 2 < 9) plus its 22 additions, the reciprocal and the
product by 1 each: a probability is off by (d + 36) eps relative.  Sums of
probabilities add positive terms over at most 44 fp32 additions and one final
rounding: (d + 81) eps, taken as (d + 96) eps with the largest d of the batch.
The gradient's terms are products of a probability (or a given weight) with sums
over the row, each (d + 36) + ln-many additions + a few roundings, bounded by
2 (d + 96) eps times the sum of the terms' magnitudes, which the oracle returns.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import synth
from gpu_cases import flush
from oracle import balance as OB
from oracle import route as OR

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_expert_ffn_router_amd as moe  # noqa: E402

DEV = torch.device("cuda")
EPS = 2.0 ** -24
MARK = -77


def _dev(a, dtype=None):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV, dtype)


class Batch:
    """One router batch: host arrays, device copies and output buffers."""

    def __init__(self, T, E, k, seq=None, masked=False, seed=0, renorm=True, logits=None):
        rng = np.random.default_rng(seed)
        self.T, self.E, self.k, self.seq, self.renorm = T, E, k, seq, renorm
        self.S = 1 if seq is None else len(seq) - 1
        self.lg = (rng.normal(size=(T, E)) * 2 + rng.normal(size=E)).astype(np.float32) \
            if logits is None else logits
        self.ids, w = OR.route(self.lg, k, renorm) if T else (np.zeros((0, k), np.int32),
                                                              np.zeros((0, k)))
        self.w = w.astype(np.float32)
        self.mask = (rng.random(T) < 0.7).astype(np.uint8) if masked else None
        self.dw = rng.normal(size=(T, k)).astype(np.float32)
        self.dl = rng.normal(size=self.S).astype(np.float32)
        self.spread = float(np.max(self.lg.max(1) - np.where(np.isfinite(self.lg), self.lg, np.inf)
                                   .min(1))) if T and np.isfinite(self.lg).any() else 0.0

    def upload(self):
        self.d = {"lg": _dev(self.lg), "ids": _dev(self.ids, torch.int32), "w": _dev(self.w),
                  "mask": _dev(self.mask), "dw": _dev(self.dw), "dl": _dev(self.dl),
                  "seq": None if self.seq is None else _dev(np.asarray(self.seq, np.int32))}
        S, E = self.S, self.E
        self.o = {"n": torch.full((S,), MARK, dtype=torch.int32, device=DEV),
                  "c": torch.full((S, E), MARK, dtype=torch.int32, device=DEV),
                  "p": torch.full((S, E), float(MARK), device=DEV),
                  "l": torch.full((S,), float(MARK), device=DEV),
                  "g": torch.full((self.T, E), float(MARK), device=DEV)}
        self.ws = torch.full((max(moe.moe_balance_loss_workspace(self.T, E, S), 16),), 0xff,
                             dtype=torch.uint8, device=DEV)
        return self

    def forward(self, stream=None):
        d, o = self.d, self.o
        moe.moe_balance_loss(d["lg"], d["ids"], self.k, o["n"], o["c"], o["p"], o["l"], self.ws,
                             d["mask"], d["seq"], stream)

    def backward(self, stream=None, weights=True, loss=True):
        d, o = self.d, self.o
        moe.moe_route_backward(d["lg"], self.k, d["ids"] if weights else None,
                               d["w"] if weights else None, d["dw"] if weights else None,
                               o["n"] if loss else None, o["c"] if loss else None,
                               d["dl"] if loss else None, o["g"], self.renorm, d["mask"], d["seq"],
                               stream)

    def check_forward(self):
        n, c, p, l = OB.balance_loss(self.lg, self.ids, self.k, self.mask, self.seq)
        o = {k: v.cpu().numpy() for k, v in self.o.items()}
        assert np.array_equal(o["n"], n) and np.array_equal(o["c"], c)
        tol = (self.spread + 96) * EPS
        assert np.all(np.abs(o["p"] - p) <= tol * p + 1e-37 * self.T)
        assert np.all(np.abs(o["l"] - l) <= tol * l)

    def check_backward(self, weights=True, loss=True):
        n, c, _, _ = OB.balance_loss(self.lg, self.ids, self.k, self.mask, self.seq)
        g, mag = OB.route_backward(self.lg, self.k, self.renorm, self.ids, self.w,
                                   self.dw if weights else None, n, c, self.dl if loss else None,
                                   np.full((self.T, self.E), float(MARK)), self.mask, self.seq)
        got = self.o["g"].cpu().numpy()
        tol = 2 * (self.spread + 96) * EPS
        assert np.all(np.abs(got - g) <= tol * mag + 1e-37)

    def run(self):
        self.upload()
        self.forward()
        self.backward()
        torch.cuda.synchronize()
        self.check_forward()
        self.check_backward()


CASES = [
    # T, E, k, seq, masked: no row; one row; one row per sequence; the sides of every row shape
    # (60/64/65, 255/256/257, 511/512/513, 1023/1024) and chunk size (128/129); empty sequences,
    # rows before the first and behind the last
    (0, 8, 2, None, False), (0, 8, 2, [0, 0, 0], False),
    (1, 1, 1, None, False), (1, 3, 2, [0, 1], False), (5, 4, 4, [0, 1, 2, 3, 4, 5], False),
    (7, 60, 4, None, True), (33, 64, 16, [3, 3, 20, 33], True), (64, 65, 3, [0, 0, 64, 64], False),
    (127, 255, 8, None, False), (128, 256, 8, [1, 100, 127], True), (129, 257, 8, [0, 128, 129], True),
    (200, 511, 5, None, False), (257, 512, 16, [5, 130, 130, 256], True), (300, 513, 2, None, True),
    (140, 1023, 9, [0, 16, 32, 140], False), (260, 1024, 16, [0, 259], True),
    (1000, 8, 2, list(range(0, 1001, 10)), True), (3001, 128, 6, [17, 400, 400, 401, 2999], True),
]


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k,seq,masked", CASES)
def test_against_oracle(T, E, k, seq, masked, renorm):
    flush(f"[router training] T={T} E={E} k={k} S={0 if seq is None else len(seq) - 1}")
    Batch(T, E, k, seq, masked, seed=T + E, renorm=renorm).run()


def test_no_row_in_many_sequences():
    Batch(0, 8, 2, [0] * 301).run()


def test_a_million_sequences():
    """2^20 sequences of which three hold rows: more slices of sums than a grid has workgroups."""
    T, E, k, S = 2000, 64, 4, 1 << 20
    small = Batch(T, E, k, [0, 700, 701, T], seed=5).upload()
    small.forward()
    seq = np.zeros(S + 1, np.int32)
    at = [3, 400_000, S - 2]                   # the sequences with rows
    seq[at[0] + 1:], seq[at[1] + 1:], seq[at[2] + 1:] = 700, 701, T
    big = Batch(T, E, k, list(seq), seed=5).upload()
    big.forward()
    big.backward()
    torch.cuda.synchronize()
    for name in "ncpl":
        got = big.o[name]
        assert torch.equal(got[at], small.o[name])
        got[at] = 0
        assert not bool(got.any())
    small.d["dl"] = big.d["dl"][at].contiguous()
    small.backward()
    torch.cuda.synchronize()
    assert torch.equal(big.o["g"], small.o["g"])


def test_every_sequence_masked():
    b = Batch(150, 40, 4, [0, 70, 150], True, seed=1)
    b.mask[:] = 0
    b.lg[:] = np.nan                           # what masked rows hold is not used
    b.ids[:] = 1 << 30
    b.spread = 0.0
    b.run()
    assert float(b.o["l"].abs().max()) == 0.0 and float(b.o["g"].abs().max()) == 0.0


@pytest.mark.parametrize("E", [8, 100, 256])
def test_masked_experts_and_masked_rows_of_anything(E):
    b = Batch(50, E, 2, [0, 20, 50], True, seed=2)
    b.lg[3, ::2] = -np.inf                     # half of the experts masked
    b.lg[4] = np.finfo(np.float32).min         # all at the type's lowest value: uniform
    b.lg[6, 1:] = np.finfo(np.float32).min     # one expert left
    b.mask[[3, 4, 6]] = 1
    b.mask[[7, 8, 9]] = 0
    b.lg[7], b.lg[8], b.lg[9] = np.nan, np.inf, -np.inf
    b.ids[7:10] = -5
    b.spread = 104.0                           # below that expf(x - m) is 0 in fp32
    b.run()


def test_row_without_any_expert():
    b = Batch(20, 12, 2, seed=3)
    b.lg[5] = -np.inf
    b.w[5], b.dw[5] = 0.0, 0.0
    b.run()
    assert float(b.o["g"][5].abs().max()) == 0.0


def test_nan_stays_in_its_sequence():
    b = Batch(300, 64, 4, [0, 100, 200, 300], seed=4).upload()
    b.d["lg"][150, 3] = float("nan")
    b.forward()
    b.backward()
    torch.cuda.synchronize()
    l, p, g = (b.o[x].cpu().numpy() for x in ("l", "p", "g"))
    assert np.isnan(l).tolist() == [False, True, False]
    assert np.all(np.isnan(p[1])) and np.all(np.isfinite(p[[0, 2]]))
    assert np.all(np.isnan(g[150])) and np.all(np.isfinite(np.delete(g, 150, 0)))


def test_dropped_and_repeated_ids():
    """Ids outside [0, E) count nowhere; an id that appears twice adds twice."""
    b = Batch(140, 20, 4, [0, 60, 140], seed=5)
    b.ids[3, 1], b.ids[4, 0], b.ids[5, 2] = -1, 20, 1 << 30
    b.ids[7] = 6
    b.ids[8, 3] = b.ids[8, 0]
    b.run()


@pytest.mark.parametrize("renorm", [True, False])
def test_parts_alone(renorm):
    b = Batch(90, 30, 3, [0, 40, 90], True, seed=6, renorm=renorm).upload()
    b.forward()
    for weights, loss in ((True, False), (False, True)):
        b.o["g"].fill_(float(MARK))
        b.backward(weights=weights, loss=loss)
        torch.cuda.synchronize()
        b.check_backward(weights, loss)


def test_gradient_against_differences():
    """The library's loss moves as its own gradient says (fixed counts)."""
    b = Batch(130, 24, 3, [0, 50, 130], seed=7)
    b.upload()
    b.forward()
    b.backward(weights=False)
    torch.cuda.synchronize()
    g = b.o["g"].double().cpu().numpy()
    n, c, _, _ = OB.balance_loss(b.lg, b.ids, b.k, None, b.seq)
    rng = np.random.default_rng(8)
    v = rng.normal(size=b.lg.shape)
    h = 1e-5

    def value(lg):
        p = OB.softmax_rows(lg)
        return sum(float(b.dl[s]) * b.E / (b.k * n[s] ** 2)
                   * np.dot(c[s], p[b.seq[s]:b.seq[s + 1]].sum(0)) for s in range(2))

    lg = b.lg.astype(np.float64)
    num = (value(lg + h * v) - value(lg - h * v)) / (2 * h)
    _, mag = OB.route_backward(b.lg, b.k, True, b.ids, b.w, None, n, c, b.dl,
                               np.zeros(b.lg.shape), None, b.seq)
    # the gradient's own tolerance along v, and the differences' h^2 term
    assert abs((g * v).sum() - num) <= 2 * (b.spread + 96) * EPS * (mag * abs(v)).sum() + 1e-7


def test_repeat_calls_and_streams_are_bit_identical():
    """No answer depends on what the workspace or the outputs held, nor on the stream."""
    b = Batch(5000, 256, 8, [0, 1000, 4800], True, seed=9).upload()
    b.forward()
    b.backward()
    torch.cuda.synchronize()
    ref = {k: v.clone() for k, v in b.o.items()}
    side = torch.cuda.Stream()
    for s in (None, side):
        for v in b.o.values():
            v.fill_(MARK)
        b.ws.fill_(0x5a)
        torch.cuda.synchronize()
        b.forward(s)
        b.backward(s)
        torch.cuda.synchronize()
        for k, v in b.o.items():
            assert torch.equal(v, ref[k]), k


def test_captured_step():
    """forward + backward in one graph, replayed on new logits with eager work between; two
    graphs with workspaces of their own."""
    bs = [Batch(T, 64, 4, [0, T // 2, T - 3], True, seed=T).upload() for T in (100, 900)]
    graphs = []
    for b in bs:
        b.forward()
        b.backward()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.forward()
            b.backward()
        graphs.append(g)
    for rep in range(3):
        for b in bs:
            new = Batch(b.T, 64, 4, b.seq, True, seed=1000 * rep + b.T)
            for name, a in (("lg", new.lg), ("ids", new.ids), ("w", new.w), ("dw", new.dw),
                            ("mask", new.mask)):
                b.d[name].copy_(torch.from_numpy(a))
                setattr(b, name, a)
            b.spread = new.spread
            for v in b.o.values():
                v.fill_(MARK)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for b in bs:
            b.check_forward()
            b.check_backward()


def test_layer_step():
    """As used: route, balance loss and both gradients through MoELayer, on a packed batch."""
    wl = synth.Workload("train", T=200, H=256, E=32, I=128, k=4, fmt="fp8_b128", seed=12)
    stride = synth.record_layout(wl.fmt, wl.H, wl.I)["stride"]
    layer = moe.MoELayer(wl.fmt, wl.E, wl.H, wl.I, wl.k, 256, stride)
    lg = synth.make_logits(wl)
    logits = torch.from_numpy(lg).to(DEV)
    layer.route_permute(logits)
    seq = torch.tensor([0, 80, 190], dtype=torch.int32, device=DEV)
    mask = (torch.arange(wl.T, device=DEV) % 7 != 0)
    bal = layer.balance_loss(logits, mask, seq)
    dw = torch.randn(wl.T * wl.k, device=DEV)
    dl = torch.tensor([0.5, -2.0], device=DEV)
    g = layer.route_backward(logits, torch.full_like(logits, float(MARK)), dw, bal, dl, mask, seq)
    torch.cuda.synchronize()
    b = Batch(wl.T, wl.E, wl.k, [0, 80, 190], logits=lg)
    b.mask = mask.cpu().numpy().astype(np.uint8)
    b.dw, b.dl = dw.cpu().numpy().reshape(wl.T, wl.k), dl.cpu().numpy()
    b.w = layer.w[:wl.T * wl.k].cpu().numpy().reshape(wl.T, wl.k)
    assert np.array_equal(layer.ids[:wl.T * wl.k].cpu().numpy().reshape(wl.T, wl.k), b.ids)
    b.o = {"n": bal["n_tokens"], "c": bal["counts"], "p": bal["probs"], "l": bal["loss"], "g": g}
    b.check_forward()
    b.check_backward()


def test_binding_refusals():
    b = Batch(10, 8, 2, [0, 10]).upload()
    d, o = b.d, b.o
    args = (d["lg"], d["ids"], 2, o["n"], o["c"], o["p"], o["l"], b.ws)
    for i, bad in ((0, d["lg"].double()), (1, d["ids"].long()), (1, d["ids"][:9]), (3, o["n"].float()),
                   (4, o["c"][:, :4]), (5, o["p"].cpu()), (6, o["l"].repeat(2)), (7, o["p"])):
        with pytest.raises(ValueError):
            moe.moe_balance_loss(*args[:i], bad, *args[i + 1:], seq_offsets=d["seq"])
    with pytest.raises(ValueError):
        moe.moe_balance_loss(*args, token_mask=d["lg"], seq_offsets=d["seq"])
    with pytest.raises(moe.MoeError):
        moe.moe_balance_loss(*args[:7], b.ws[:16], seq_offsets=d["seq"])


@pytest.mark.parametrize("T,E,S", [(100, 16, 3000), (100, 300, 257), (5000, 16, 70000), (300, 100, 5000)])
def test_many_empty_sequences(T, E, S):
    """Far more sequences than rows: runs of empty ones are searched past, not walked."""
    rng = np.random.default_rng(T + S)
    seq = np.sort(rng.integers(0, T + 1, S + 1)).astype(np.int32)
    seq[S // 3:S // 3 + S // 4] = seq[S // 3]          # one long run of empty sequences
    seq = np.sort(seq)
    b = Batch(T, E, 3, None, True, seed=S)
    b.seq, b.S = seq, S
    b.dl = rng.normal(size=S).astype(np.float32)
    b.run()


def test_largest_row_and_k():
    b = Batch(400, 1024, 16, [0, 399], seed=21)
    b.lg[7] = 0.0                                       # every expert equal
    b.run()


def test_two_calls_at_once():
    """Two batches on two streams, each with its workspace: the results of each alone."""
    bs = [Batch(T, 200, 4, [0, T // 3, T], True, seed=T).upload() for T in (3000, 2500)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for b, s in zip(bs, streams):
            b.forward(s)
            b.backward(s)
    torch.cuda.synchronize()
    for b in bs:
        b.check_forward()
        b.check_backward()
