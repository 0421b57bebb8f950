"""The operators that train the experts of the MoE layer as measured cases.

Six calls, each in a plain form (elementary torch operations in 32 bits or
more) and as the library's call:

  dispatch       moe_dispatch             token rows into expert order
  dispatch_grad  moe_dispatch_backward    its gradient: each token's k rows summed back
  combine_grad   moe_combine_backward     gradient of the weighted combine
  ffn_train      moe_expert_ffn_train     SwiGLU FFN of every expert over its rows, keeping
                                          the gate and up products for the gradient
  ffn_grad       moe_expert_ffn_backward  gradients of the rows and of every expert's weights
  clip           moe_clip_grad_norm       norm over all gradients, and the gradients clipped

Definitions (t token, j < k, a = t k + j, inv[a] the assignment's row in expert order,
w[a] its routing weight, e the expert of row p):
  dispatch       x_perm[inv[a]] = w[a] x[t]                       (w absent: 1)
  dispatch_grad  d_x[t] = sum_j w[a] d_x_perm[inv[a]] + d_add[t];  d_w[a] = <d_x_perm[inv[a]], x[t]>
  combine_grad   d_y_perm[inv[a]] = w[a] dy[t];                    d_w[a] = <y_perm[inv[a]], dy[t]>
  ffn_train      g = Wg[e] x[p], u = Wu[e] x[p];  y[p] = Wd[e] (silu(g) u)
  ffn_grad       from g, u and dy:  dh = Wd[e]^T dy[p], s = 1 / (1 + e^-g), du = dh g s,
                 dg = dh u s (1 + g (1 - s));  dx[p] = Wg[e]^T dg + Wu[e]^T du;
                 dWg[e] = sum_p dg x[p]^T, dWu[e] = sum_p du x[p]^T, dWd[e] = sum_p dy[p] (g s u)^T
  clip           norm = sqrt(sum of all squares);  scale = min(1, max_norm / (norm + 1e-6));
                 out_i = scale grad_i
Gate and up stand side by side: w13 [E][2I][H] (gate rows, then up rows), gate_up [A][2I].
"""
import math

import torch

own = False

DEV = "cuda"
BF16 = torch.bfloat16


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the tokens of one decode batch, copied into expert order for another device
        dict(name="dispatch_decode_batch", op="dispatch", T=8, H=2048, E=256, k=8, weighted=False),
        # a large training batch of the widest layer, weights applied on the way in
        dict(name="dispatch_large_batch", op="dispatch", T=16384, H=7168, E=256, k=8, weighted=True),
        # the same way back on a short batch (odd token count), weights learned
        dict(name="dispatch_grad_small", op="dispatch_grad", T=333, H=2048, E=60, k=4,
             weighted=True, add=False),
        # a large batch; the gradient of the shared expert is added on the way
        dict(name="dispatch_grad_large_batch", op="dispatch_grad", T=16384, H=4096, E=512, k=8,
             weighted=False, add=True),
        # the smallest layer
        dict(name="combine_grad_small", op="combine_grad", T=64, H=256, E=8, k=2),
        # a large training batch of the widest layer
        dict(name="combine_grad_large_batch", op="combine_grad", T=16384, H=7168, E=256, k=8),
        # the smallest layer
        dict(name="ffn_train_small", op="ffn_train", T=64, H=256, I=128, E=8, k=2),
        # a training batch: about 512 rows an expert, ragged
        dict(name="ffn_train_batch", op="ffn_train", T=4096, H=2048, I=1024, E=64, k=8),
        # a fine-tuning batch of a small layer: odd everything
        dict(name="ffn_grad_small", op="ffn_grad", T=777, H=1024, I=384, E=13, k=3),
        # a training batch: about 2048 rows an expert, ragged
        dict(name="ffn_grad_batch", op="ffn_grad", T=16384, H=4096, I=1024, E=64, k=8),
        # routers and norms of a stack of layers: many small tensors
        dict(name="clip_many_small", op="clip", n=60, least=256, most=16384, floats=1.0),
        # the experts' weights (bf16) and routers of a layer stack
        dict(name="clip_experts", op="clip", n=12, least=4096, most=1 << 29, floats=0.25),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_grad", "combine_grad", "ffn_train", "ffn_train", "ffn_grad",
                     "ffn_grad", "clip"])
    if op in ("dispatch", "dispatch_grad", "combine_grad"):
        E = _log_int(rng, 2, 512)
        k = rng.randint(1, min(E, 8))
        H = 8 * _log_int(rng, 4, 896)
        T = _log_int(rng, 1, 16384)
        case = dict(op=op, T=T, H=H, E=E, k=k)
        if op != "combine_grad":
            case["weighted"] = rng.random() < 0.5
        if op == "dispatch_grad":
            case["add"] = rng.random() < 0.5
        return case
    if op == "clip":
        least = _log_int(rng, 1, 100000)
        return dict(op=op, n=rng.randint(1, 60), least=least, most=least * _log_int(rng, 1, 200),
                    floats=rng.choice([0.0, 0.5, 1.0]))
    E = _log_int(rng, 1, 64)
    k = rng.randint(1, min(E, 8))
    H, I = 128 * _log_int(rng, 1, 32), 128 * _log_int(rng, 1, 8)
    return dict(op=op, T=_log_int(rng, 1, 4096), H=H, I=I, E=E, k=k)


def _sizes(case):
    """Elements of every gradient: geometrically from least to most, every second one a whole
    multiple of 1024, the others as they fall."""
    n, lo, hi = case["n"], case["least"], case["most"]
    sizes = [int(lo * (hi / lo) ** (i / max(n - 1, 1))) for i in range(n)]
    return [max(1024, s // 1024 * 1024) if i % 2 else s for i, s in enumerate(sizes)]


def _is_float(case, i):
    """Which gradients are fp32 (the others bf16): the smallest ones, as routers and norms are."""
    return i < case["floats"] * case["n"]


def work(case):
    op = case["op"]
    if op == "clip":
        b = [(4 if _is_float(case, i) else 2) * s for i, s in enumerate(_sizes(case))]
        return {"bytes": 2 * sum(b) + 8, "flops": 3 * sum(_sizes(case))}
    T, H, k = case["T"], case["H"], case["k"]
    A = T * k
    if op == "dispatch":
        return {"bytes": T * H * 2 + A * H * 2 + A * 4 + A * 4 * case["weighted"],
                "flops": A * H * case["weighted"]}
    if op == "dispatch_grad":
        return {"bytes": A * H * 2 + T * H * 2 + A * 4 + T * H * 2 * case["add"]
                + (A * 8 + T * H * 2) * case["weighted"],
                "flops": A * H * (4 if case["weighted"] else 1)}
    if op == "combine_grad":
        return {"bytes": 2 * A * H * 2 + T * H * 2 + A * 12, "flops": 3 * A * H}
    E, I = case["E"], case["I"]
    touched = min(E, A)
    if op == "ffn_train":
        return {"bytes": touched * 3 * H * I * 2 + T * H * 2 + A * (2 * I + H) * 2 + A * 4
                + (2 * E + 1) * 4, "flops": 6 * A * H * I}
    return {"bytes": touched * 3 * H * I * 2 + E * 3 * H * I * 2 + T * H * 2 + A * (2 * I + 2 * H) * 2
            + A * 4 + (2 * E + 1) * 4, "flops": 12 * A * H * I}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _routing(T, E, k, g):
    """A routed batch of a layer with a few favoured experts: weights [T][k], counts [E],
    offsets [E+1], sorted_idx [A], inv_idx [A]."""
    logits = torch.randn(T, E, generator=g, device=DEV) * 1.5
    logits += torch.randn(E, generator=g, device=DEV) * 0.7
    top, ids = torch.topk(logits, k, dim=1)
    ids = ids.reshape(-1)
    counts = torch.zeros(E, dtype=torch.int64, device=DEV).scatter_add_(0, ids, torch.ones_like(ids))
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), counts.cumsum(0)])
    order = torch.argsort(ids, stable=True)
    inv = torch.empty_like(order)
    inv[order] = torch.arange(order.numel(), device=DEV)
    i32 = [t.to(torch.int32).contiguous() for t in (counts, offsets, order, inv)]
    return [torch.softmax(top, 1).contiguous()] + i32


def _rows(n, H, g, size=1.0):
    # rows of unit size with a few large channels
    out = torch.empty(n, H, dtype=BF16, device=DEV)
    ch = torch.exp(0.5 * torch.randn(H, generator=g, device=DEV)) * size
    for r in range(0, n, 8192):
        m = min(8192, n - r)
        out[r:r + m] = torch.randn(m, H, generator=g, device=DEV) * ch
    return out


def _weight(E, N, K, g):
    out = torch.empty(E, N, K, dtype=BF16, device=DEV)
    for e in range(E):
        out[e] = torch.randn(N, K, generator=g, device=DEV) * K ** -0.5
    return out


def _package():
    import moe_expert_ffn_router_amd as moe
    return moe


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 6007 + 29)
    op = case["op"]
    st = {"case": dict(case)}
    if op == "clip":
        # gradients of very different sizes; the norm is a few times the bound
        st["grads"], st["out"] = [], []
        for i, n in enumerate(_sizes(case)):
            dt = torch.float32 if _is_float(case, i) else BF16
            t = torch.empty(n, dtype=dt, device=DEV)
            size = 1e-3 * 2.0 ** (i % 7)
            for r in range(0, n, 1 << 26):
                m = min(1 << 26, n - r)
                t[r:r + m] = torch.randn(m, generator=g, device=DEV) * size
            st["grads"].append(t)
            st["out"].append(torch.empty_like(t))
        st["max_norm"] = 0.01 * math.sqrt(sum(_sizes(case))) * 0.1
        st["norm_scale"] = torch.zeros(2, device=DEV)
        if own:
            moe = _package()
            st["ws"] = torch.empty(moe.moe_clip_grad_norm_workspace(case["n"]), dtype=torch.uint8,
                                   device=DEV)
        return st
    T, H, E, k = case["T"], case["H"], case["E"], case["k"]
    A = T * k
    st["w"], st["counts"], st["offsets"], st["sorted_idx"], st["inv"] = _routing(T, E, k, g)
    if op == "dispatch":
        st["x"] = _rows(T, H, g)
        st["x_perm"] = torch.zeros(A, H, dtype=BF16, device=DEV)
    elif op == "dispatch_grad":
        st["d_x_perm"] = _rows(A, H, g, 0.01)
        st["x"] = _rows(T, H, g)
        st["add"] = _rows(T, H, g, 0.01) if case["add"] else None
        st["d_x"] = torch.zeros(T, H, dtype=BF16, device=DEV)
        st["dw"] = torch.zeros(T, k, device=DEV)
    elif op == "combine_grad":
        st["dy"] = _rows(T, H, g, 0.01)
        st["y_perm"] = _rows(A, H, g)
        st["d_y_perm"] = torch.zeros(A, H, dtype=BF16, device=DEV)
        st["dw"] = torch.zeros(T, k, device=DEV)
    else:
        I = case["I"]
        # one record an expert: w13 and w2 one behind the other (both whole multiples of 256 bytes)
        w13, w2 = _weight(E, 2 * I, H, g), _weight(E, H, I, g)
        st["base"] = torch.cat([w13.view(E, -1), w2.view(E, -1)], 1).contiguous()
        st["x"] = _rows(T, H, g)
        st["cap"] = int(st["counts"].max())
        if op == "ffn_train":
            st["gate_up"] = torch.zeros(A, 2 * I, dtype=BF16, device=DEV)
            st["y_perm"] = torch.zeros(A, H, dtype=BF16, device=DEV)
        else:
            st["gate_up"] = _rows(A, 2 * I, g)
            st["dy"] = _rows(A, H, g, 0.01)
            st["d_x_perm"] = torch.zeros(A, H, dtype=BF16, device=DEV)
            st["d_w13"] = torch.zeros(E, 2 * I, H, dtype=BF16, device=DEV)
            st["d_w2"] = torch.zeros(E, H, I, dtype=BF16, device=DEV)
        if own:
            moe = _package()
            st["W"] = moe.experts("bf16", E, H, I, st["base"], st["base"].shape[1] * 2)
            size = (moe.moe_expert_ffn_train_workspace if op == "ffn_train"
                    else moe.moe_expert_ffn_backward_workspace)(st["W"], T, k)
            st["ws"] = torch.empty(max(size, 256), dtype=torch.uint8, device=DEV)
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _dispatch_plain(st):
    k, order = st["case"]["k"], st["sorted_idx"].long()
    rows = st["x"].float()[order // k]
    if st["case"]["weighted"]:
        rows = rows * st["w"].reshape(-1)[order][:, None]
    return rows.to(BF16)


def _dispatch_grad_plain(st):
    T, H, k = (st["case"][n] for n in ("T", "H", "k"))
    rows = st["d_x_perm"].float()[st["inv"].long()].view(T, k, H)
    dx = (rows * st["w"][:, :, None] if st["case"]["weighted"] else rows).sum(1)
    if st["add"] is not None:
        dx = dx + st["add"].float()
    if not st["case"]["weighted"]:
        return dx.to(BF16)
    return dx.to(BF16), (rows * st["x"].float()[:, None, :]).sum(2)


def _combine_grad_plain(st):
    T, H, k = (st["case"][n] for n in ("T", "H", "k"))
    order, dy = st["sorted_idx"].long(), st["dy"].float()
    rows = dy[order // k] * st["w"].reshape(-1)[order][:, None]
    y = st["y_perm"].float()[st["inv"].long()].view(T, k, H)
    return rows.to(BF16), (y * dy[:, None, :]).sum(2)


def _weights(st):
    E, H, I = (st["case"][n] for n in ("E", "H", "I"))
    b = st["base"]
    return b[:, :2 * I * H].reshape(E, 2 * I, H), b[:, 2 * I * H:].reshape(E, H, I)


def _slots(st):
    """Row numbers [E, cap] of every expert's rows, and which of them exist."""
    i = torch.arange(st["cap"], device=DEV)
    rows = st["offsets"][:-1, None].long() + i
    live = i < st["counts"][:, None]
    return torch.where(live, rows, 0), live


def _spread(rows, slots):
    """Rows in expert order as [E, cap, n] in fp32, zeros where an expert has fewer."""
    return torch.where(slots[1][:, :, None], rows[slots[0]].float(), 0.0)


def _gather(padded, slots, A):
    """The rows of [E, cap, n] back in expert order, in bf16."""
    out = torch.zeros(A, padded.shape[2], dtype=BF16, device=DEV)
    out[slots[0][slots[1]]] = padded[slots[1]].to(BF16)
    return out


def _ffn_train_plain(st):
    T, I, k = (st["case"][n] for n in ("T", "I", "k"))
    w13, w2 = _weights(st)
    slots = _slots(st)
    x = _spread(st["x"][st["sorted_idx"].long() // k], slots)
    gu = torch.bmm(x, w13.float().transpose(1, 2))
    g, u = gu[:, :, :I], gu[:, :, I:]
    h = g / (1.0 + torch.exp(-g)) * u
    y = torch.bmm(h, w2.float().transpose(1, 2))
    return _gather(gu, slots, T * k), _gather(y, slots, T * k)


def _ffn_grad_plain(st):
    T, I, k = (st["case"][n] for n in ("T", "I", "k"))
    w13, w2 = _weights(st)
    slots = _slots(st)
    x = _spread(st["x"][st["sorted_idx"].long() // k], slots)
    gu, dy = _spread(st["gate_up"], slots), _spread(st["dy"], slots)
    g, u = gu[:, :, :I], gu[:, :, I:]
    s = 1.0 / (1.0 + torch.exp(-g))
    dh = torch.bmm(dy, w2.float())
    d_w2 = torch.bmm(dy.transpose(1, 2), g * s * u)
    dgu = torch.cat([dh * u * s * (1.0 + g * (1.0 - s)), dh * g * s], 2)
    dx = torch.bmm(dgu, w13.float())
    d_w13 = torch.bmm(dgu.transpose(1, 2), x)
    return _gather(dx, slots, T * k), d_w13.to(BF16), d_w2.to(BF16)


def _clip_plain(st):
    total = torch.stack([t.float().square().sum(dtype=torch.float64) for t in st["grads"]]).sum()
    norm = total.sqrt()
    scale = (st["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    return norm.float(), scale, [(t.float() * scale).to(t.dtype) for t in st["grads"]]


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own(st):
    moe = _package()
    case = st["case"]
    op, k = case["op"], case.get("k")
    if op == "dispatch":
        moe.moe_dispatch(st["x"], st["inv"], k, st["x_perm"],
                         topk_w=st["w"] if case["weighted"] else None)
        return st["x_perm"]
    if op == "dispatch_grad":
        if not case["weighted"]:
            moe.moe_dispatch_backward(st["d_x_perm"], st["inv"], k, st["d_x"], d_add=st["add"])
            return st["d_x"]
        moe.moe_dispatch_backward(st["d_x_perm"], st["inv"], k, st["d_x"], topk_w=st["w"],
                                  d_add=st["add"], x=st["x"], d_topk_w=st["dw"])
        return st["d_x"], st["dw"]
    if op == "combine_grad":
        moe.moe_combine_backward(st["dy"], st["inv"], st["w"], k, st["d_y_perm"],
                                 y_perm=st["y_perm"], d_topk_w=st["dw"])
        return st["d_y_perm"], st["dw"]
    if op == "ffn_train":
        moe.moe_expert_ffn_train(st["W"], st["x"], case["T"], k, st["counts"], st["offsets"],
                                 st["sorted_idx"], st["gate_up"], st["y_perm"], st["ws"])
        return st["gate_up"], st["y_perm"]
    if op == "ffn_grad":
        moe.moe_expert_ffn_backward(st["W"], st["x"], case["T"], k, st["counts"], st["offsets"],
                                    st["sorted_idx"], st["gate_up"], st["dy"], st["ws"],
                                    d_x_perm=st["d_x_perm"], d_w13=st["d_w13"], d_w2=st["d_w2"])
        return st["d_x_perm"], st["d_w13"], st["d_w2"]
    moe.moe_clip_grad_norm(st["grads"], st["max_norm"], st["norm_scale"], st["ws"],
                           clipped=st["out"])
    return st["norm_scale"][0], st["norm_scale"][1], st["out"]


_PLAIN = {"dispatch": _dispatch_plain, "dispatch_grad": _dispatch_grad_plain,
          "combine_grad": _combine_grad_plain, "ffn_train": _ffn_train_plain,
          "ffn_grad": _ffn_grad_plain, "clip": _clip_plain}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# the same from the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "clip":
        squares = sum(float(torch.dot(c, c)) for t in st["grads"]
                      for c in (p.double() for p in t.split(1 << 26)))
        norm = math.sqrt(squares)
        scale = min(1.0, st["max_norm"] / (norm + 1e-6))
        one = lambda v: torch.tensor(v, dtype=torch.float64, device=DEV)  # noqa: E731
        return one(norm), one(scale), [t.double().mul_(scale) for t in st["grads"]]
    T, H, k = case["T"], case["H"], case["k"]
    w, inv = st["w"].double(), st["inv"].long().view(T, k)
    if op in ("dispatch", "combine_grad"):
        src = st["x"] if op == "dispatch" else st["dy"]
        out = torch.empty(T * k, H, dtype=torch.float64, device=DEV)
        dw = torch.empty(T, k, dtype=torch.float64, device=DEV)
        for j in range(k):
            wj = w[:, j, None] if case.get("weighted", True) else 1.0
            out[inv[:, j]] = src.double() * wj
            if op == "combine_grad":
                dw[:, j] = torch.linalg.vecdot(st["y_perm"][inv[:, j]].double(), src.double())
        return out if op == "dispatch" else (out, dw)
    if op == "dispatch_grad":
        dx = torch.zeros(T, H, dtype=torch.float64, device=DEV) if st["add"] is None else st["add"].double()
        dw = torch.empty(T, k, dtype=torch.float64, device=DEV)
        for j in range(k):
            r = st["d_x_perm"][inv[:, j]].double()
            dx += r * w[:, j, None] if case["weighted"] else r
            dw[:, j] = torch.linalg.vecdot(r, st["x"].double())
        return (dx, dw) if case["weighted"] else dx
    I, E = case["I"], case["E"]
    w13, w2 = _weights(st)
    ends, tok = st["offsets"].tolist(), st["sorted_idx"].long() // k
    f64 = dict(dtype=torch.float64, device=DEV)
    if op == "ffn_train":
        gate_up, y = torch.zeros(T * k, 2 * I, **f64), torch.zeros(T * k, H, **f64)
    else:
        dx = torch.zeros(T * k, H, **f64)
        d_w13, d_w2 = torch.zeros(E, 2 * I, H, **f64), torch.zeros(E, H, I, **f64)
    for e in range(E):
        p = slice(ends[e], ends[e + 1])
        if p.start == p.stop:
            continue
        x = st["x"][tok[p]].double()
        if op == "ffn_train":
            g, u = x @ w13[e, :I].double().t(), x @ w13[e, I:].double().t()
            gate_up[p, :I], gate_up[p, I:] = g, u
            y[p] = (torch.sigmoid(g) * g * u) @ w2[e].double().t()
            continue
        g, u = st["gate_up"][p, :I].double(), st["gate_up"][p, I:].double()
        dy = st["dy"][p].double()
        sig = torch.sigmoid(g)
        dh = dy @ w2[e].double()
        du, dg = dh * g * sig, dh * u * (sig + g * sig * (1.0 - sig))
        dx[p] = dg @ w13[e, :I].double() + du @ w13[e, I:].double()
        d_w13[e, :I], d_w13[e, I:] = dg.t() @ x, du.t() @ x
        d_w2[e] = dy.t() @ (g * sig * u)
    return (gate_up, y) if op == "ffn_train" else (dx, d_w13, d_w2)
