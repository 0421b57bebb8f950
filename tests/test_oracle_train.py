"""CPU pins of the training oracle, and what the training calls refuse before they touch a device."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

from oracle import combine as OC
from oracle import permute as OP
from oracle import train as OT

m = pytest.importorskip("moe_expert_ffn_router_amd")


def _case(T=7, k=2, E=4, H=6, I=5, seed=0):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    counts, offsets, sorted_idx, inv = OP.permute(ids, E)[:4]
    return dict(rng=rng, T=T, k=k, E=E, H=H, I=I, ids=ids, offsets=np.asarray(offsets),
                sorted_idx=np.asarray(sorted_idx).ravel(), inv=np.asarray(inv).ravel(),
                x=rng.normal(size=(T, H)), w=rng.random((T, k)), w13=rng.normal(size=(E, 2 * I, H)),
                w2=rng.normal(size=(E, H, I)), r=rng.normal(size=(T, H)))


def _forward(c, x=None, w=None, w13=None, w2=None):
    x = c["x"] if x is None else x
    rows, _ = OT.dispatch(x, c["inv"], None, c["T"] * c["k"])
    _, _, y = OT.ffn_train(rows, c["offsets"], c["w13"] if w13 is None else w13,
                           c["w2"] if w2 is None else w2)
    return OC.combine(y, c["inv"], c["w"] if w is None else w, c["T"], c["k"])


def _backward(c):
    rows, _ = OT.dispatch(c["x"], c["inv"], None, c["T"] * c["k"])
    gu, _, y = OT.ffn_train(rows, c["offsets"], c["w13"], c["w2"])
    d_y_perm, d_w = OT.combine_backward(c["r"], y, c["inv"], c["w"])
    d_rows, d_w13, d_w2 = OT.ffn_backward(rows, c["offsets"], c["w13"], c["w2"], gu, d_y_perm)
    d_x, _ = OT.dispatch_backward(d_rows, c["inv"], None, c["x"])
    return {"x": d_x, "w": d_w, "w13": d_w13, "w2": d_w2}


@pytest.mark.parametrize("name", ["x", "w", "w13", "w2"])
def test_gradients_are_central_differences(name):
    c = _case()
    grad = _backward(c)[name]
    base, h = c[name], 1e-5
    for flat in c["rng"].choice(base.size, size=min(base.size, 25), replace=False):
        up, dn = base.copy(), base.copy()
        up.flat[flat] += h
        dn.flat[flat] -= h
        d = ((_forward(c, **{name: up}) - _forward(c, **{name: dn})) * c["r"]).sum() / (2 * h)
        assert d == pytest.approx(grad.flat[flat], rel=1e-6, abs=1e-7)


def test_dispatch_weights_by_differences_and_adjoint():
    c = _case(seed=1)
    R = c["T"] * c["k"]
    r = c["rng"].normal(size=(R, c["H"]))
    out, named = OT.dispatch(c["x"], c["inv"], c["w"], R)
    assert named.all()
    d_x, d_w = OT.dispatch_backward(r, c["inv"], c["w"], c["x"])
    assert (out * r).sum() == pytest.approx((c["x"] * d_x).sum(), rel=1e-12)
    assert (out * r).sum() == pytest.approx((c["w"] * d_w).sum(), rel=1e-12)  # linear in w
    add = c["rng"].normal(size=c["x"].shape)
    assert np.allclose(OT.dispatch_backward(r, c["inv"], c["w"], c["x"], add)[0], d_x + add)


def test_dropped_assignments_have_no_row():
    c = _case(seed=2)
    R = c["T"] * c["k"]
    inv = c["inv"].copy()
    inv[3], inv[8] = -1, R
    out, named = OT.dispatch(c["x"], inv, c["w"], R)
    assert not named[c["inv"][3]] and not named[c["inv"][8]] and not out[c["inv"][3]].any()
    _, d_w = OT.dispatch_backward(np.ones((R, c["H"])), inv, None, c["x"])
    assert d_w.ravel()[3] == 0 and d_w.ravel()[8] == 0 and (d_w != 0).sum() == R - 2


def test_a_rows_weight_gradient_alone():
    """Weight gradients are sums over rows: those of each row alone add up to the whole."""
    c = _case(T=1, k=1, E=1, seed=3)
    rng = c["rng"]
    x, gu, dy = rng.normal(size=(5, 6)), rng.normal(size=(5, 10)), rng.normal(size=(5, 6))
    whole = OT.ffn_backward(x, [0, 5], c["w13"], c["w2"], gu, dy)
    parts = [OT.ffn_backward(x[i:i + 1], [0, 1], c["w13"], c["w2"], gu[i:i + 1], dy[i:i + 1])
             for i in range(5)]
    assert np.allclose(whole[1], sum(p[1] for p in parts)) and np.allclose(whole[2], sum(p[2] for p in parts))
    assert np.allclose(whole[0], np.concatenate([p[0] for p in parts]))


def test_clip():
    n, s, c = OT.clip_grad_norm([np.array([3.0]), np.array([[0.0, 4.0]])], 1.0)
    assert n == 5.0 and s == pytest.approx(0.2, rel=1e-6) and np.allclose(c[1], [[0, 0.8]], rtol=1e-6)
    assert OT.clip_grad_norm([np.array([3.0])], 4.0)[1] == 1.0


# ---------------------------------------------------------------------------
# refusals: addresses that are never touched
# ---------------------------------------------------------------------------
L = m._lib
P = 4096          # an aligned address
BAD_ARG, UNSUPPORTED, WORKSPACE = m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED, m.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), BAD_ARG), (dict(k=0), BAD_ARG), (dict(k=17), BAD_ARG), (dict(H=12), BAD_ARG),
    (dict(H=0), BAD_ARG), (dict(R=-1), BAD_ARG), (dict(src=None), BAD_ARG), (dict(inv=None), BAD_ARG),
    (dict(out=None), BAD_ARG), (dict(src=P + 2), BAD_ARG), (dict(w=P + 4), BAD_ARG),
    (dict(T=1 << 27, k=2), UNSUPPORTED), (dict(R=(1 << 27) + 1), UNSUPPORTED)])
def test_row_calls_refuse(over, status):
    a = dict(T=4, k=2, H=64, R=8, src=P, inv=P, w=P, out=P) | over
    sizes = (a["T"], a["k"], a["H"], a["R"])
    assert L.moe_dispatch(a["src"], a["inv"], a["w"], *sizes, a["out"], None) == status
    assert L.moe_dispatch_backward(a["src"], a["inv"], a["w"], None, *sizes, None, a["out"], None,
                                   None) == status
    assert L.moe_combine_backward(a["src"], None, a["inv"], a["w"], *sizes, a["out"], None, None) == status


def test_row_calls_refuse_dots_without_their_rows():
    assert L.moe_dispatch_backward(P, P, P, None, 4, 2, 64, 8, None, P, P, None) == BAD_ARG
    assert L.moe_combine_backward(P, None, P, P, 4, 2, 64, 8, P, P, None) == BAD_ARG
    assert L.moe_combine_backward(P, P, P, None, 4, 2, 64, 8, P, None, None) == BAD_ARG
    assert b"moe_combine_backward" in L.moe_last_error()


def _experts(**over):
    a = dict(fmt=0, E=4, H=256, I=128, base=P, stride=256 * 128 * 6) | over
    return m.Experts(a["fmt"], a["E"], a["H"], a["I"], a["base"], a["stride"])


BIG = 1 << 40   # workspace bytes, said but not used


@pytest.mark.parametrize("W,over,status", [
    (dict(fmt=1), {}, UNSUPPORTED), (dict(H=200), {}, UNSUPPORTED), (dict(I=64), {}, UNSUPPORTED),
    (dict(E=0), {}, BAD_ARG), (dict(E=1025), {}, BAD_ARG), (dict(stride=256), {}, BAD_ARG),
    (dict(base=None), {}, BAD_ARG), ({}, dict(T=-1), BAD_ARG), ({}, dict(k=0), BAD_ARG),
    ({}, dict(k=17), BAD_ARG), ({}, dict(x=None), BAD_ARG), ({}, dict(x=P + 8), BAD_ARG),
    ({}, dict(counts=None), BAD_ARG), ({}, dict(offsets=None), BAD_ARG),
    ({}, dict(sorted_idx=P + 4), BAD_ARG), ({}, dict(gate_up=None), BAD_ARG),
    ({}, dict(rows=None), BAD_ARG), ({}, dict(ws=None), BAD_ARG), ({}, dict(ws_bytes=100), WORKSPACE),
    ({}, dict(T=1 << 24, k=16), UNSUPPORTED), ({}, dict(T=1 << 23, k=1), UNSUPPORTED)])
def test_ffn_calls_refuse(W, over, status):
    W = _experts(**W)
    a = dict(T=8, k=2, x=P, counts=P, offsets=P, sorted_idx=P, gate_up=P, rows=P, ws=P,
             ws_bytes=BIG) | over
    head = (ctypes.byref(W), a["x"], a["T"], a["k"], a["counts"], a["offsets"], a["sorted_idx"], a["gate_up"],
            a["rows"])
    assert L.moe_expert_ffn_train(*head, a["ws"], a["ws_bytes"], None) == status
    assert L.moe_expert_ffn_backward(*head, P, P, P, 0, 0, a["ws"], a["ws_bytes"], None) == status


def test_ffn_backward_refuses_gradient_types():
    W = _experts()
    call = lambda t, acc, d=P: L.moe_expert_ffn_backward(  # noqa: E731
        ctypes.byref(W), P, 8, 2, P, P, P, P, P, P, d, P, t, acc, P, BIG, None)
    assert call(2, 0) == UNSUPPORTED and call(-1, 0) == UNSUPPORTED
    assert call(0, 1) == UNSUPPORTED          # bf16 gradients do not accumulate
    assert call(1, 1, P + 4) == BAD_ARG
    assert L.moe_expert_ffn_backward(None, P, 8, 2, P, P, P, P, P, P, P, P, 0, 0, P, BIG, None) == BAD_ARG


def _clip(grads, numel, types, out, max_norm=1.0, ws_bytes=BIG, ns=P, ws=P):
    n = len(grads)
    arr = lambda t, v: None if v is None else (t * n)(*v)  # noqa: E731
    return L.moe_clip_grad_norm(n, arr(ctypes.c_void_p, grads), arr(ctypes.c_int64, numel),
                                arr(ctypes.c_int32, types), max_norm, arr(ctypes.c_void_p, out), ns, ws,
                                ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(grads=[P], numel=[8], types=[2], out=None), UNSUPPORTED),
    (dict(grads=[P], numel=[-1], types=[0], out=None), BAD_ARG),
    (dict(grads=[None], numel=[8], types=[0], out=None), BAD_ARG),
    (dict(grads=[P + 2], numel=[8], types=[1], out=None), BAD_ARG),
    (dict(grads=[P + 1], numel=[8], types=[0], out=None), BAD_ARG),
    (dict(grads=[P], numel=[8], types=[0], out=[None]), BAD_ARG),
    (dict(grads=[P], numel=[8], types=[0], out=[P], max_norm=-1.0), BAD_ARG),
    (dict(grads=[P], numel=[8], types=[0], out=[P], max_norm=float("nan")), BAD_ARG),
    (dict(grads=[P], numel=[8], types=[0], out=[P], ns=None), BAD_ARG),
    (dict(grads=[P], numel=[8], types=[0], out=[P], ws=None), BAD_ARG),
    (dict(grads=[P], numel=[8], types=[0], out=[P], ws_bytes=64), WORKSPACE),
    # the same gradient twice, clipped in place; overlapping outputs; an output over a gradient
    (dict(grads=[P, P], numel=[8, 8], types=[0, 0], out=[P, P]), BAD_ARG),
    (dict(grads=[P, 2 * P], numel=[8, 8], types=[0, 0], out=[3 * P, 3 * P + 14]), BAD_ARG),
    (dict(grads=[P, 2 * P], numel=[8, 8], types=[0, 0], out=[2 * P + 8, 3 * P]), BAD_ARG),
    (dict(grads=[P], numel=[8], types=[0], out=[P + 2]), BAD_ARG)])
def test_clip_refuses(kw, status):
    assert _clip(**kw) == status


def test_workspace_queries():
    W = _experts()
    up = lambda v: -(-v // 256) * 256  # noqa: E731
    for T, two in ((7, 14), (48, 96), (700, 96)):  # rows that are held in two parts, or may be in a smaller batch
        A = 2 * T
        h, dgu = up(A * 128 * 2) + up(two * 128 * 2), up(A * 256 * 2) + up(two * 256 * 2)
        assert m.moe_expert_ffn_train_workspace(W, T, 2) == h
        assert m.moe_expert_ffn_backward_workspace(W, T, 2) == h + dgu
    assert m.moe_expert_ffn_train_workspace(W, -1, 2) == 0
    assert m.moe_clip_grad_norm_workspace(1) >= 8 and m.moe_clip_grad_norm_workspace(-1) == 0
    assert m.moe_clip_grad_norm_workspace(1 << 16) >= m.moe_clip_grad_norm_workspace(129)
