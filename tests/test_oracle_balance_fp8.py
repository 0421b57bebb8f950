"""Pins of the balance-loss, routing-gradient and FP8-product oracles (CPU), planted
mistakes in them, and the refusals of the library's calls (no GPU touched)."""
import ctypes

import numpy as np
import pytest
import torch

import synth
from oracle import balance as OB
from oracle import formats as OF
from oracle import fp8 as O8
from oracle import route as OR

m = pytest.importorskip("moe_expert_ffn_router_amd")


# ---- balance loss ----------------------------------------------------------
def test_uniform_router_has_loss_one():
    T, E, k = 24, 8, 2
    ids = np.arange(T * k).reshape(T, k) % E          # every expert equally often
    n, c, p, loss = OB.balance_loss(np.zeros((T, E)), ids, k)
    assert n[0] == T and np.all(c == T * k // E) and np.allclose(p, T / E)
    assert abs(loss[0] - 1.0) < 1e-14


def test_collapsed_router():
    T, E, k = 10, 5, 1
    lg = np.zeros((T, E))
    lg[:, 3] = 60.0
    loss = OB.balance_loss(lg, np.full((T, k), 3), k)[3]
    assert abs(loss[0] - E) < 1e-12


def test_masked_and_empty_sequences():
    rng = np.random.default_rng(0)
    T, E, k = 20, 6, 2
    lg = rng.normal(size=(T, E)).astype(np.float32)
    ids, _ = OR.route(lg, k)
    mask = np.ones(T, np.uint8)
    mask[4:9] = 0
    lg[5] = np.nan                                    # masked rows hold anything
    ids[6] = 999
    seq = [2, 4, 9, 9, 18]                            # the second is masked, the third empty
    n, c, p, loss = OB.balance_loss(lg, ids, k, mask, seq)
    assert n.tolist() == [2, 0, 0, 9]
    assert np.all(c[1:3] == 0) and np.all(p[1:3] == 0) and np.all(loss[1:3] == 0)
    alone = OB.balance_loss(lg[9:18], ids[9:18], k)
    assert np.array_equal(c[3], alone[1][0]) and np.allclose(p[3], alone[2][0], rtol=1e-14)
    assert np.isclose(loss[3], alone[3][0], rtol=1e-14)


def test_row_without_experts_counts_nothing():
    lg = np.full((2, 4), -np.inf)
    lg[1] = [0.0, -np.inf, 0.0, -np.inf]
    p = OB.balance_loss(lg, np.zeros((2, 1), int), 1)[2][0]
    assert p.tolist() == [0.5, 0.0, 0.5, 0.0]


def _loss_and_weights(lg, ids, k, renorm, counts, coef_w, coef_l, seq, mask):
    """coef_l . loss(fixed counts) + coef_w . weights, the function whose gradient is taken."""
    T, E = lg.shape
    p = OB.softmax_rows(lg)
    total = 0.0
    for s in range(len(seq) - 1):
        r = np.arange(seq[s], seq[s + 1])
        r = r[mask[r].astype(bool)]
        if len(r):
            total += coef_l[s] * E / (k * len(r) ** 2) * np.dot(counts[s], p[r].sum(0))
        for t in r:
            sel = lg[t, ids[t]].astype(np.float64)
            w = np.exp(sel - sel.max())
            w = w / w.sum() if renorm else p[t, ids[t]]
            total += np.dot(coef_w[t], w)
    return total


@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(renorm):
    rng = np.random.default_rng(3)
    T, E, k = 9, 7, 3
    lg = rng.normal(size=(T, E))
    ids, w = OR.route(lg.astype(np.float32), k, renorm)
    p = OB.softmax_rows(lg)
    sel = np.take_along_axis(lg, ids.astype(np.int64), 1)
    w = np.exp(sel - sel.max(1, keepdims=True))
    w = w / w.sum(1, keepdims=True) if renorm else np.take_along_axis(p, ids.astype(np.int64), 1)
    mask = np.ones(T, np.uint8)
    mask[[2, 6]] = 0
    seq = [0, 4, 4, 8]                                # the last row belongs to no sequence
    n, c, _, _ = OB.balance_loss(lg, ids, k, mask, seq)
    cl, cw = rng.normal(size=3), rng.normal(size=(T, k))
    before = rng.normal(size=(T, E))
    g, mag = OB.route_backward(lg, k, renorm, ids, w, cw, n, c, cl, before, mask, seq)
    assert np.array_equal(g[8], before[8]) and np.all(g[[2, 6]] == 0)
    assert np.all(mag[:8] >= np.abs(g[:8]) - 1e-15)
    h = 1e-6
    for t in range(8):
        for e in range(E):
            up, dn = lg.copy(), lg.copy()
            up[t, e] += h
            dn[t, e] -= h
            args = (ids, k, renorm, c, cw, cl, seq, mask)
            d = (_loss_and_weights(up, *args) - _loss_and_weights(dn, *args)) / (2 * h)
            assert abs(d - g[t, e]) < 1e-8 * max(1.0, mag[t, e]), (t, e, d, g[t, e])


def test_planted_balance_mistakes_are_caught(monkeypatch):
    right = OB.route_backward

    def no_inner(lg, k, renorm, ids, w, dw, n, c, dl, before, mask=None, seq=None):
        g, mag = right(lg, k, True, ids, w, dw, n, c, dl, before, mask, seq)
        return g, mag                                  # renormalised form for both

    monkeypatch.setattr(OB, "route_backward", no_inner)
    with pytest.raises(AssertionError):
        test_gradient_against_differences(False)
    monkeypatch.undo()
    loss = OB.balance_loss
    monkeypatch.setattr(OB, "balance_loss",
                        lambda *a, **kw: loss(*a, **kw)[:3] + (loss(*a, **kw)[3] * 1.5,))
    with pytest.raises(AssertionError):
        test_uniform_router_has_loss_one()


# ---- FP8 -------------------------------------------------------------------
def test_every_code_round_trips():
    v = OF.e4m3_value(np.arange(127)).astype(np.float64)
    x = np.zeros((2, 128))
    x[0, :127], x[1, :127] = v, -v                     # the block maximum is 448: scale 1
    codes, scales = O8.quantize(x)
    assert np.all(scales == 1.0)
    assert codes[0, :127].tolist() == list(range(127))
    assert np.array_equal(O8.decode(codes), x)


def test_quantize_against_torch_cast_and_ties():
    rng = np.random.default_rng(5)
    x = rng.normal(size=(4, 300)) * np.exp(rng.normal(size=(4, 300)) * 3)
    x[0, :5] = [448.0, 17.0, 19.0, -21.0, 2.0 ** -10]  # 17, 19 tie; 2^-10 ties with zero
    x[0, 5:128] = 0
    codes, scales = O8.quantize(x.astype(np.float32))
    assert codes[0, 1] == 0x58 and codes[0, 2] == 0x5a and codes[0, 4] == 0
    t = torch.from_numpy(x.astype(np.float32))
    s = torch.from_numpy(np.repeat(scales, 128, 1)[:, :300]).float()
    ref = (t / s).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(codes, ref)


def test_scale_edges():
    assert O8.scale_of(448.0) == 1.0 and O8.scale_of(448.0 * (1 + 2.0 ** -7)) == 2.0
    assert O8.scale_of(224.0) == 0.5 and O8.scale_of(0.0) == 1.0
    assert O8.scale_of(2.0 ** -133) == 2.0 ** -126
    assert np.isnan(O8.scale_of(float("inf"))) and np.isnan(O8.scale_of(float("nan")))


def test_product_against_scalar_loop():
    rng = np.random.default_rng(6)
    M, N, K = 3, 130, 144
    a, w = rng.integers(0, 127, (M, K)).astype(np.uint8), rng.integers(0, 127, (N, K)).astype(np.uint8)
    sa, sw = rng.random((M, 2)), rng.random((2, 2))
    y, mag = O8.matmul(a, sa, w, sw)
    for i in range(M):
        for j in (0, 127, 128, 129):
            t = sum(OF.e4m3_value(a[i, q]) * sa[i, q // 128] * OF.e4m3_value(w[j, q])
                    * sw[j // 128, q // 128] for q in range(K))
            assert abs(t - y[i, j]) <= 1e-12 * mag[i, j]


def test_planted_fp8_mistakes_are_caught(monkeypatch):
    scale = O8.scale_of
    monkeypatch.setattr(O8, "scale_of", lambda a: scale(a) * 2 if a == 448.0 else scale(a))
    with pytest.raises(AssertionError):
        test_every_code_round_trips()
    monkeypatch.undo()
    monkeypatch.setattr(O8, "weight_value", lambda c, s: O8.decode(c) * s[0, 0])
    with pytest.raises(AssertionError):
        test_product_against_scalar_loop()


# ---- refusals of the C ABI (arguments are checked before anything is enqueued) ----
P = 4096  # a non-null, aligned address that is never dereferenced


def _refused(status, name, *args):
    assert getattr(m._lib, name)(*args) == status, (name, args, m._lib.moe_last_error())
    if status != m.MOE_OK:
        assert name.encode() in m._lib.moe_last_error()


def test_balance_loss_refusals():
    f, big = "moe_balance_loss", 1 << 30

    def args(logits=P, ids=P, T=4, E=8, k=2, mask=None, seq=None, S=1, n=P, c=P, p=P, loss=P, ws=P,
             nb=big):
        return (logits, ids, T, E, k, mask, seq, S, n, c, p, loss, ws, nb, None)

    for bad in (dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(E=64, k=17),
                dict(S=0), dict(S=2), dict(seq=P, S=(1 << 20) + 1), dict(logits=None),
                dict(ids=None), dict(n=None), dict(c=None), dict(p=None), dict(loss=None),
                dict(ws=None), dict(logits=P + 4), dict(ids=P + 4), dict(mask=P + 1),
                dict(seq=P + 4), dict(n=P + 4), dict(c=P + 4), dict(p=P + 4), dict(loss=P + 4),
                dict(ws=P + 8)):
        _refused(m.MOE_ERR_INVALID_ARG, f, *args(**bad))
    _refused(m.MOE_ERR_UNSUPPORTED, f, *args(T=(1 << 27) + 1))
    need = m.moe_balance_loss_workspace(4, 8, 1)
    assert need > 0
    _refused(m.MOE_ERR_WORKSPACE, f, *args(nb=need - 1))
    assert m.moe_balance_loss_workspace(-1, 8, 1) == m.moe_balance_loss_workspace(4, 0, 1) == 0


def test_route_backward_refusals():
    f = "moe_route_backward"

    def args(logits=P, T=4, E=8, k=2, ids=P, w=P, dw=P, mask=None, seq=None, S=1, n=P, c=P, dl=P,
             out=P):
        return (logits, T, E, k, 1, ids, w, dw, mask, seq, S, n, c, dl, out, None)

    for bad in (dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(S=0), dict(S=3),
                dict(logits=None), dict(out=None), dict(ids=None), dict(w=None), dict(n=None),
                dict(c=None), dict(dw=None, dl=None), dict(logits=P + 4), dict(out=P + 4),
                dict(ids=P + 4), dict(w=P + 4), dict(dw=P + 4), dict(n=P + 4), dict(c=P + 4),
                dict(dl=P + 4), dict(mask=P + 2), dict(seq=P + 4)):
        _refused(m.MOE_ERR_INVALID_ARG, f, *args(**bad))
    _refused(m.MOE_ERR_UNSUPPORTED, f, *args(T=(1 << 27) + 1))
    _refused(m.MOE_OK, f, *args(T=0, logits=None, out=None))


def test_fp8_refusals():
    q = "moe_fp8_quantize"
    for bad in ((P, -1, 64, P, P), (P, 4, 0, P, P), (P, 4, 12, P, P), (P, 4, 65544, P, P),
                (None, 4, 64, P, P), (P, 4, 64, None, P), (P, 4, 64, P, None), (P + 2, 4, 64, P, P),
                (P, 4, 64, P + 8, P), (P, 4, 64, P, P + 4)):
        _refused(m.MOE_ERR_INVALID_ARG, q, *bad, None)
    _refused(m.MOE_OK, q, None, 0, 64, None, None, None)

    def args(a=P, sa=P, M=4, w=P, sw=P, N=32, K=64, c=None, o=None, E=1, y=P, ws=P, nb=1 << 30):
        return (a, sa, M, w, sw, N, K, c, o, E, y, ws, nb, None)

    f = "moe_fp8_matmul"
    for bad in (dict(M=-1), dict(N=0), dict(K=0), dict(K=24), dict(N=65537), dict(K=65552),
                dict(E=0), dict(E=1025, c=P, o=P), dict(E=2), dict(c=P), dict(o=P), dict(a=None),
                dict(sa=None), dict(w=None), dict(sw=None), dict(y=None), dict(a=P + 8),
                dict(sa=P + 4), dict(w=P + 8), dict(sw=P + 4), dict(y=P + 2), dict(ws=P + 8),
                dict(c=P + 4, o=P), dict(c=P, o=P + 4)):
        _refused(m.MOE_ERR_INVALID_ARG, f, *args(**bad))
    _refused(m.MOE_ERR_UNSUPPORTED, f, *args(N=65536, K=65536))
    _refused(m.MOE_ERR_UNSUPPORTED, f, *args(M=(1 << 27) + 1))
    _refused(m.MOE_OK, f, *args(M=0, a=None, y=None))


def test_expert_ffn_fp8_refusals():
    f = "moe_expert_ffn_fp8"
    st = synth.record_layout("fp8_b128", 256, 128)["stride"]

    def args(fmt="fp8_b128", E=8, H=256, I=128, stride=st, base=P, x=P, T=4, k=2, c=P, o=P, s=P, y=P,
             ws=P, nb=1 << 30, slot=None):
        W = m.experts(fmt, E, H, I, base, stride)
        return (ctypes.byref(W), slot, x, T, k, c, o, s, y, ws, nb, None)

    for bad in (dict(E=0), dict(E=1025), dict(base=None), dict(base=P + 8), dict(stride=st - 256),
                dict(stride=st + 8), dict(T=-1), dict(k=0), dict(k=9), dict(E=64, k=17),
                dict(x=None), dict(c=None), dict(o=None), dict(s=None), dict(y=None), dict(ws=None),
                dict(x=P + 2), dict(c=P + 4), dict(o=P + 4), dict(s=P + 4), dict(y=P + 2),
                dict(ws=P + 4), dict(slot=P + 4)):
        _refused(m.MOE_ERR_INVALID_ARG, f, *args(**bad))
    _refused(m.MOE_ERR_INVALID_ARG, f, None, *args()[1:])
    for fmt in ("bf16", "mxfp4", "nvfp4"):
        _refused(m.MOE_ERR_UNSUPPORTED, f, *args(fmt=fmt, stride=1 << 20))
    _refused(m.MOE_ERR_UNSUPPORTED, f, *args(H=200, stride=1 << 20))
    _refused(m.MOE_ERR_UNSUPPORTED, f, *args(T=1 << 27))
    # rows past 32-bit offsets on 16-row tiles, more of them than a grid can hold
    _refused(m.MOE_ERR_UNSUPPORTED, f, *args(
        T=1 << 20, H=4096, I=16384, k=8, nb=1 << 62,
        stride=synth.record_layout("fp8_b128", 4096, 16384)["stride"]))
    W = m.experts("fp8_b128", 8, 256, 128, P, st)
    need = m.moe_expert_ffn_fp8_workspace(W, 4, 2)
    assert 0 < need <= m.moe_expert_ffn_fp8_workspace(W, 5, 2)
    W2 = m.experts("fp8_b128", 8, 2048, 512, P, st)     # never less for more tokens
    sizes = [m.moe_expert_ffn_fp8_workspace(W2, T, 2) for T in range(0, 2000, 7)]
    assert sizes == sorted(sizes)
    _refused(m.MOE_ERR_WORKSPACE, f, *args(nb=need - 1))
    _refused(m.MOE_OK, f, *args(T=0))


def test_binding_refuses_host_and_mistyped_tensors():
    lg = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="device tensor"):
        m.moe_balance_loss(lg, lg, 2, lg, lg, lg, lg, lg)
    with pytest.raises(ValueError, match="matrix"):
        m.moe_fp8_quantize(torch.zeros(4), lg, lg)
    with pytest.raises(TypeError):
        m._arg(3, "x", torch.float32, None, lg.device)
    with pytest.raises(ValueError, match="dtype"):
        m._arg(lg, "x", torch.int32, None, lg.device)
    with pytest.raises(ValueError, match="elements"):
        m._arg(lg, "x", torch.float32, 31, lg.device)
    with pytest.raises(ValueError, match="contiguous"):
        m._arg(lg.t(), "x", torch.float32, None, lg.device)
