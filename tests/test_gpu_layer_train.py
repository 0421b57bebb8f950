"""A training step of the layer on the GPU: MoELayer.forward_train and backward against the
formulas in 64 bits on the same routing, with clipping behind them.

Tolerances.  Along each path independent roundings to bf16 (at most b = 2^-8 relative each, so
b / sqrt(3) of a result's norm, and less than 1.5 times that for a thousand elements) add in
squares; a kept gate or up product enters the gradient's sums through a factor of at most 1.1
relative to them.  The number of roundings on each path is given with each check.
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
B = 2.0 ** -8


def near(got, want, roundings, what):
    rel = float((got.double() - want).norm() / want.norm())
    assert rel <= 1.5 * math.sqrt(roundings) * B / math.sqrt(3), (what, rel)


class Step:
    def __init__(self, T, E, H, I, k, shared_I=0, seed=0, T_max=None):
        g = torch.Generator(device=DEV).manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
        self.T, self.E, self.H, self.I, self.k, self.shared_I = T, E, H, I, k, shared_I
        self.logits = rnd(T, E) * 1.5
        self.x, self.d_y = rnd(T, H).to(BF), (rnd(T, H) * 0.1).to(BF)

        def weights(n, i):
            w13, w2 = (rnd(n, 2 * i, H) * H ** -0.5).to(BF), (rnd(n, H, i) * i ** -0.5).to(BF)
            return w13, w2, torch.cat([w13.view(n, -1), w2.view(n, -1)], 1).contiguous()

        self.w13, self.w2, self.rec = weights(E, I)
        stride = moe.moe_expert_layout_query("bf16", H, I)["stride"]
        ss = moe.moe_expert_layout_query("bf16", H, shared_I)["stride"] if shared_I else 0
        self.layer = moe.MoELayer("bf16", E, H, I, k, T_max or T, stride, shared_I, ss)
        self.W = self.layer.weights(self.rec)
        self.Ws = None
        if shared_I:
            self.s13, self.s2, self.srec = weights(1, shared_I)
            self.Ws = moe.experts("bf16", 1, H, shared_I, self.srec, ss)

    def grads(self, dtype):
        z = lambda *s: torch.full(s, 7.0, dtype=dtype, device=DEV)  # noqa: E731
        r = dict(d_w13=z(self.E, 2 * self.I, self.H), d_w2=z(self.E, self.H, self.I))
        if self.shared_I:
            r |= dict(d_s13=z(1, 2 * self.shared_I, self.H), d_s2=z(1, self.H, self.shared_I))
        return r

    def run(self, dtype=BF, stream=None, d_loss=None):
        y = self.layer.forward_train(self.logits, self.x, self.W, self.Ws, stream=stream)
        g = self.grads(dtype)
        bal = self.layer.balance_loss(self.logits, stream=stream) if d_loss is not None else None
        r = self.layer.backward(self.logits, self.x, self.W, self.d_y, Ws=self.Ws, balance=bal,
                                d_loss=d_loss, stream=stream, **g)
        return y, g | r

    def exact(self, d_loss=None):
        """(y, gradients) by differentiating the formulas in 64 bits, on the layer's own choice of
        experts."""
        ids = self.layer.ids[:self.T * self.k].view(self.T, self.k).long()
        t = lambda a: a.double().requires_grad_(True)  # noqa: E731
        v = dict(logits=t(self.logits), x=t(self.x), w13=t(self.w13), w2=t(self.w2))
        if self.shared_I:
            v |= dict(s13=t(self.s13), s2=t(self.s2))
        w = torch.softmax(v["logits"].gather(1, ids), 1)
        w.retain_grad()

        def ffn(x, w13, w2):
            z = x @ w13.t()
            i = z.shape[1] // 2
            return (z[:, :i] * torch.sigmoid(z[:, :i]) * z[:, i:]) @ w2.t()

        y = torch.zeros(self.T, self.H, dtype=torch.float64, device=DEV)
        for e in range(self.E):
            tok, j = (ids == e).nonzero(as_tuple=True)
            if tok.numel():
                y = y.index_add(0, tok, ffn(v["x"][tok], v["w13"][e], v["w2"][e]) * w[tok, j][:, None])
        if self.shared_I:
            y = y + ffn(v["x"], v["s13"][0], v["s2"][0])
        loss = (y * self.d_y.double()).sum()
        if d_loss is not None:
            c = torch.bincount(ids.reshape(-1), minlength=self.E).double()
            p = torch.softmax(v["logits"], 1).sum(0)
            loss = loss + float(d_loss[0]) * self.E / (self.k * self.T ** 2) * (c * p).sum()
        loss.backward()
        r = {"d_" + n: a.grad for n, a in v.items()}
        r["d_topk_w"] = w.grad
        return y.detach(), r


SIZES = [dict(T=64, E=8, H=256, I=128, k=2), dict(T=333, E=13, H=512, I=384, k=3, shared_I=256),
         dict(T=100, E=3, H=128, I=256, k=3), dict(T=1, E=8, H=256, I=128, k=2, shared_I=128),
         dict(T=700, E=60, H=256, I=256, k=4, T_max=900)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: f"T{s['T']}E{s['E']}")
def test_step(size, dtype):
    flush(f"[layer train] {size} {dtype}")
    s = Step(**size)
    d_loss = torch.tensor([0.3], device=DEV)
    y, g = s.run(dtype, d_loss=d_loss)
    want_y, want = s.exact(d_loss)
    near(y, want_y, 4, "y")                          # h, y_perm, (y_shared,) y
    for n in ("d_w13", "d_w2", "d_s13", "d_s2"):
        if n in g:
            near(g[n], want[n], 6, n)                # d_y_perm, g, u (1.1 each), (dg; du) or h, result
    near(g["d_x"], want["d_x"], 8, "d_x")            # the same, d_x_perm, the shared expert's, d_x
    if size["T"] > 1:
        near(g["d_topk_w"], want["d_topk_w"], 4, "d_topk_w")   # h, y_perm
        near(g["d_logits"], want["d_logits"], 5, "d_logits")   # differences of the former
    # all gradients clipped together, in place
    ts = [g[n] for n in g if n not in ("d_x", "d_topk_w")]
    norm = math.sqrt(sum(float(t.double().square().sum()) for t in ts))
    ns = torch.empty(2, device=DEV)
    ws = torch.empty(moe.moe_clip_grad_norm_workspace(len(ts)), dtype=torch.uint8, device=DEV)
    moe.moe_clip_grad_norm(ts, norm / 3, ns, ws, clipped=ts)
    assert float(ns[0]) == pytest.approx(norm, rel=1e-6)
    after = math.sqrt(sum(float(t.double().square().sum()) for t in ts))
    assert after == pytest.approx(norm / 3, rel=2 * B)


def test_accumulated_micro_batches():
    """Two halves of a batch, their weight gradients added in fp32, against the whole batch's."""
    s = Step(T=128, E=8, H=256, I=128, k=2, seed=3)
    _, whole = s.run(F32)
    acc = s.grads(F32)
    for t in acc.values():
        t.zero_()
    for half in (slice(0, 64), slice(64, 128)):
        lg, x = s.logits[half].contiguous(), s.x[half].contiguous()
        s.layer.forward_train(lg, x, s.W)
        r = s.layer.backward(lg, x, s.W, s.d_y[half].contiguous(), accumulate=True, **acc)
        assert torch.equal(r["d_x"], whole["d_x"][half])
    for n in acc:
        # only the order of fp32 sums differs: at most 64 additions of each half and one more
        assert float((acc[n] - whole[n]).norm() / whole[n].norm()) <= 130 * 2.0 ** -24


def test_backward_twice_and_on_a_stream():
    s = Step(T=200, E=8, H=256, I=256, k=2, shared_I=128, seed=4)
    y, first = s.run()
    y = y.clone()
    again = s.grads(BF)
    r = s.layer.backward(s.logits, s.x, s.W, s.d_y, Ws=s.Ws, **again)
    assert all(torch.equal(first[n], v) for n, v in (again | r).items())
    st = torch.cuda.Stream()
    other = Step(T=200, E=8, H=256, I=256, k=2, shared_I=128, seed=4)
    torch.cuda.synchronize()
    y2, g2 = other.run(stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(y2, y) and all(torch.equal(first[n], g2[n]) for n in first)


def test_no_tokens():
    s = Step(T=0, E=4, H=128, I=128, k=2, T_max=8)
    y = s.layer.forward_train(s.logits, s.x, s.W)
    g = s.grads(BF)
    r = s.layer.backward(s.logits, s.x, s.W, s.d_y, **g)
    assert y.shape[0] == 0 and r["d_x"].shape == (0, 128) and not g["d_w13"].any() and not g["d_w2"].any()


def test_captured_step():
    """Forward, backward and clipping in one graph; every replay equals the eager step."""
    s = Step(T=96, E=8, H=256, I=128, k=2, seed=5)
    _, g = s.run(F32)
    ts = [g["d_w13"], g["d_w2"]]
    ns = torch.empty(2, device=DEV)
    ws = torch.empty(moe.moe_clip_grad_norm_workspace(2), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = s.layer.forward_train(s.logits, s.x, s.W)
        r = s.layer.backward(s.logits, s.x, s.W, s.d_y, d_w13=ts[0], d_w2=ts[1])
        moe.moe_clip_grad_norm(ts, 0.5, ns, ws, clipped=ts)
    for i in range(3):
        s.x.copy_(torch.randn(s.x.shape, device=DEV).to(BF))
        s.logits.copy_(torch.randn(s.logits.shape, device=DEV))
        graph.replay()
        got = [t.clone() for t in (y, r["d_x"], r["d_logits"], ts[0], ts[1], ns)]
        ey, eg = s.run(F32)
        ets, ens = [eg["d_w13"], eg["d_w2"]], torch.empty(2, device=DEV)
        moe.moe_clip_grad_norm(ets, 0.5, ens, ws, clipped=ets)
        for a, b in zip(got, (ey, eg["d_x"], eg["d_logits"], *ets, ens)):
            assert torch.equal(a, b)


def test_forward_train_is_the_layers_forward():
    s = Step(T=64, E=8, H=256, I=128, k=2, seed=6)
    y = s.layer.forward_train(s.logits, s.x, s.W).clone()
    near(s.layer.forward(s.logits, s.x, s.W), y.double(), 6, "y")


def test_backward_refuses_what_was_not_kept():
    """Backward wants the forward_train of the same tokens, with the shared expert alike, and no other
    call on the layer since that wrote what it kept."""
    s = Step(T=32, E=8, H=256, I=128, k=2, shared_I=128, seed=7, T_max=64)
    back = lambda **kw: s.layer.backward(**(dict(logits=s.logits, x=s.x, W=s.W, d_y=s.d_y, Ws=s.Ws)  # noqa: E731
                                            | s.grads(BF) | kw))
    with pytest.raises(ValueError):
        back()
    fwd = lambda: s.layer.forward_train(s.logits, s.x, s.W, s.Ws)  # noqa: E731
    fwd()
    back()
    for kw in (dict(logits=s.logits[:31], x=s.x[:31], d_y=s.d_y[:31]), dict(Ws=None), dict(x=s.x[:31]),
               dict(d_y=s.d_y[:, :128]), dict(x=s.x.view(16, 512))):
        with pytest.raises(ValueError):
            back(**kw)
    s.layer.balance_loss(s.logits)
    s.layer.combine(32, True)
    back()
    for other in (lambda: s.layer.forward(s.logits[:8], s.x[:8], s.W), lambda: s.layer.route(s.logits[:8]),
                  lambda: s.layer.route_permute(s.logits), lambda: s.layer.expert_ffn(s.W, s.x, 32)):
        fwd()
        back()
        other()
        with pytest.raises(ValueError):
            back()
