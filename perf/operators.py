"""The router-training and FP8 operators as measured cases.

Five operators of the MoE layer, each in a plain form (elementary torch
operations in 32 bits or more) and as the library's call:

  balance     moe_balance_loss    load-balance loss of each packed sequence,
                                  per-expert counts and probability sums
  route_grad  moe_route_backward  gradient of the routing weights and of the
                                  balance loss with respect to the logits
  quantize    moe_fp8_quantize    bf16 rows -> E4M3 with one power-of-two
                                  scale per 128 columns
  matmul      moe_fp8_matmul      E4M3 x E4M3 product with block scales, dense
                                  or grouped by expert
  ffn         moe_expert_ffn_fp8  per-expert SwiGLU FFN on FP8 records with
                                  E4M3 activations

Definitions (t token, e expert, s sequence, v_t = 1 for tokens that count):
  p[t] = softmax(logits[t]);  n_s = sum v_t;  c_se = #{(t, j): v_t, ids[t,j] = e}
  P_se = sum_t v_t p[t,e];    loss_s = E / (k n_s^2) sum_e c_se P_se  (0 if n_s = 0)
  quantize: scale = the least power of two >= amax / 448 (at least 2^-126; 1
  for a block of zeros), code = E4M3 nearest-even of x / scale
  matmul: y = bf16( sum_b a_scale[m,b] w_scale[n/128,b] sum_{k in b} a[m,k] w[n,k] )
"""
import math

import torch

own = False

DEV = "cuda"
QMAX = 448.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode batch of a serving engine that watches its router's balance
        dict(name="balance_decode_batch", op="balance", T=64, E=256, k=8, S=1, masked=False),
        # a packed training batch: ragged sequences, padding tokens masked out
        dict(name="balance_packed_batch", op="balance", T=16384, E=256, k=8, S=13, masked=True),
        # router tuning on a short batch of a small layer (odd token count)
        dict(name="route_grad_small", op="route_grad", T=333, E=60, k=4, S=3, renorm=False,
             masked=False),
        # router tuning on a large packed batch of a 512-expert layer
        dict(name="route_grad_packed_batch", op="route_grad", T=65536, E=512, k=8, S=29,
             renorm=True, masked=True),
        # the rows of one decode batch
        dict(name="quantize_decode_rows", op="quantize", T=8, K=2048),
        # a prefill batch of the widest layer
        dict(name="quantize_prefill_rows", op="quantize", T=16384, K=7168),
        # a single token through a dense projection
        dict(name="matmul_one_token", op="matmul", M=1, N=7168, K=2048, E=0),
        # ragged everything: rows, output columns and a short last K block
        dict(name="matmul_ragged", op="matmul", M=777, N=1413, K=2000, E=0),
        # a prefill batch through a dense projection
        dict(name="matmul_prefill", op="matmul", M=8192, N=4096, K=7168, E=0),
        # the gate/up product of a batch over 64 experts
        dict(name="matmul_grouped", op="matmul", M=16384, N=2048, K=4096, E=64),
        # a decode batch: at most eight experts per token, few rows each
        dict(name="ffn_decode_batch", op="ffn", T=8, H=2048, I=512, E=256, k=8),
        # a prefill batch
        dict(name="ffn_prefill_batch", op="ffn", T=4096, H=2048, I=1024, E=64, k=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "route_grad", "quantize", "matmul", "matmul", "ffn", "ffn"])
    if op in ("balance", "route_grad"):
        E = _log_int(rng, 4, 1024)
        k = rng.randint(1, min(E, 16))
        T = _log_int(rng, 1, min(65536, 65536 * 512 // E))
        S = min(_log_int(rng, 1, 64), T)
        case = dict(op=op, T=T, E=E, k=k, S=S, masked=rng.random() < 0.5)
        if op == "route_grad":
            case["renorm"] = rng.random() < 0.5
        return case
    if op == "quantize":
        K = 8 * _log_int(rng, 2, 2048)
        return dict(op=op, T=_log_int(rng, 1, min(16384, 16384 * 7168 // K)), K=K)
    if op == "matmul":
        E = rng.choice([0, 0, 2, 7, 32, 64])
        K, N = 16 * _log_int(rng, 4, 256 if E else 448), _log_int(rng, 16, 2048 if E else 4096)
        M = _log_int(rng, 1, 8192)
        return dict(op=op, M=M, N=N, K=K, E=E)
    E = rng.choice([4, 13, 32, 64])
    return dict(op=op, T=_log_int(rng, 1, 4096), H=128 * rng.randint(1, 16),
                I=128 * rng.randint(1, 8), E=E, k=rng.randint(1, min(E, 8)))


def _up(v, a):
    return (v + a - 1) // a * a


def work(case):
    op = case["op"]
    if op == "balance":
        T, E, k, S = (case[n] for n in ("T", "E", "k", "S"))
        return {"bytes": T * E * 4 + T * k * 4 + (T if case["masked"] else 0) + S * E * 8 + S * 12,
                "flops": T * E * 4}
    if op == "route_grad":
        T, E, k, S = (case[n] for n in ("T", "E", "k", "S"))
        return {"bytes": T * E * 8 + T * k * 12 + (T if case["masked"] else 0) + S * E * 4 + S * 12,
                "flops": T * E * 7}
    if op == "quantize":
        T, K = case["T"], case["K"]
        return {"bytes": T * K * 3 + T * (_up(K, 128) // 128) * 4, "flops": T * K * 2}
    if op == "matmul":
        M, N, K, E = (case[n] for n in ("M", "N", "K", "E"))
        touched = min(max(E, 1), M) if E else 1
        nb, kb = _up(N, 128) // 128, _up(K, 128) // 128
        return {"bytes": M * K + M * kb * 4 + touched * (N * K + nb * kb * 4) + M * N * 2
                + (2 * E + 1) * 4 * bool(E), "flops": 2 * M * N * K}
    T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
    touched = min(E, T * k)
    record = 3 * H * I + 3 * (H // 128) * (I // 128) * 4
    return {"bytes": touched * record + T * H * 2 + T * k * H * 2 + T * k * 4 + (2 * E + 1) * 4,
            "flops": 2 * T * k * 3 * H * I}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _logits(T, E, g):
    # router logits of a layer with a few favoured experts
    bias = torch.randn(E, generator=g, device=DEV) * 0.7
    return torch.randn(T, E, generator=g, device=DEV) * 1.5 + bias


def _topk(logits, k, renorm=True):
    v, ids = torch.topk(logits, k, dim=1)
    w = torch.softmax(v, 1) if renorm else torch.softmax(logits, 1).gather(1, ids)
    return ids.to(torch.int32).contiguous(), w.contiguous()


def _sequences(T, S, g):
    # S sequences packed into the batch, a few rows of padding behind the last
    used = T - min(T // 50, 97)
    cuts = torch.sort(torch.randint(0, used + 1, (S - 1,), generator=g, device=DEV)).values
    z = torch.zeros(1, dtype=torch.int64, device=DEV)
    return torch.cat([z, cuts, z + used]).to(torch.int32)


def _groups(rows, E, k, g):
    """Routed assignments of rows tokens: counts, offsets, sorted_idx (int32)."""
    ids = _topk(_logits(rows, E, g), k)[0].reshape(-1).to(torch.int64)
    counts = torch.zeros(E, dtype=torch.int64, device=DEV).scatter_add_(0, ids, torch.ones_like(ids))
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), counts.cumsum(0)])
    sorted_idx = torch.argsort(ids, stable=True)
    i32 = lambda t: t.to(torch.int32).contiguous()  # noqa: E731
    return i32(counts), i32(offsets), i32(sorted_idx)


def _fp8_codes(shape, g):
    # E4M3 codes of a block-quantised matrix: most values well inside the range
    out = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
    flat = out.view(-1, shape[-1])
    step = max(1, (1 << 26) // shape[-1])
    for r in range(0, flat.shape[0], step):
        n = min(step, flat.shape[0] - r)
        t = torch.randn(n, shape[-1], generator=g, device=DEV) * 90.0
        flat[r:r + n] = t.clamp(-QMAX, QMAX).to(torch.float8_e4m3fn)
    return out


def _layout(H, I):
    """Byte offsets of an FP8 expert record's sections, and the record stride."""
    w13 = 0
    w13s = _up(w13 + 2 * I * H, 256)
    w2 = _up(w13s + (2 * I // 128) * (H // 128) * 4, 256)
    w2s = _up(w2 + H * I, 256)
    return w13, w13s, w2, w2s, _up(w2s + (H // 128) * (I // 128) * 4, 256)


def _package():
    import moe_expert_ffn_router_amd as moe
    return moe


def prepare(case, seed):
    g = _gen(case, seed)
    op = case["op"]
    st = {"case": dict(case)}
    if op in ("balance", "route_grad"):
        T, E, k, S = (case[n] for n in ("T", "E", "k", "S"))
        st["logits"] = _logits(T, E, g)
        st["ids"], st["w"] = _topk(st["logits"], k, case.get("renorm", True))
        st["seq"] = _sequences(T, S, g)
        st["mask"] = ((torch.rand(T, generator=g, device=DEV) < 0.9).to(torch.uint8)
                      if case["masked"] else None)
        st["n"] = torch.zeros(S, dtype=torch.int32, device=DEV)
        st["counts"] = torch.zeros(S, E, dtype=torch.int32, device=DEV)
        if op == "balance":
            st["probs"] = torch.zeros(S, E, device=DEV)
            st["loss"] = torch.zeros(S, device=DEV)
        else:
            v, q = _valid(st)
            st["n"].copy_(_seq_sum(v.to(torch.int64), st["seq"]))
            st["counts"].copy_(_counts(st, v, q))
            st["dw"] = torch.randn(T, k, generator=g, device=DEV) * 0.05
            st["dloss"] = torch.rand(S, generator=g, device=DEV) * 0.02
            st["dlogits"] = torch.zeros(T, E, device=DEV)
    elif op == "quantize":
        T, K = case["T"], case["K"]
        # activations: unit rows with a few large channels, some rows of padding zeros
        ch = torch.exp(torch.randn(K, generator=g, device=DEV))
        x = torch.randn(T, K, generator=g, device=DEV) * ch
        x[5::17] = 0.0
        st["x"] = x.to(torch.bfloat16)
        st["codes"] = torch.zeros(T, K, dtype=torch.float8_e4m3fn, device=DEV)
        st["scales"] = torch.zeros(T, _up(K, 128) // 128, device=DEV)
    elif op == "matmul":
        M, N, K, E = (case[n] for n in ("M", "N", "K", "E"))
        kb, nb = _up(K, 128) // 128, _up(N, 128) // 128
        st["a"] = _fp8_codes((M, K), g)
        st["sa"] = torch.exp2(torch.randint(-9, -4, (M, kb), generator=g, device=DEV).float())
        lead = (E,) if E else ()
        st["w_"] = _fp8_codes(lead + (N, K), g)
        st["sw"] = 2e-4 * (0.5 + torch.rand(lead + (nb, kb), generator=g, device=DEV))
        st["y"] = torch.zeros(M, N, dtype=torch.bfloat16, device=DEV)
        st["counts"] = st["offsets"] = None
        if E:
            st["counts"], st["offsets"], _ = _groups(M, E, 1, g)
            st["cap"] = int(st["counts"].max())
    else:
        T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
        o13, o13s, o2, o2s, stride = _layout(H, I)
        base = torch.zeros(E, stride, dtype=torch.uint8, device=DEV)
        for off, n_, k_ in ((o13, 2 * I, H), (o2, H, I)):
            codes = _fp8_codes((E, n_, k_), g)
            base[:, off:off + n_ * k_] = codes.view(torch.uint8).reshape(E, -1)
        for off, n_, k_ in ((o13s, 2 * I, H), (o2s, H, I)):
            s = 2.2e-4 * (0.5 + torch.rand(E, (n_ // 128) * (k_ // 128), generator=g, device=DEV))
            base[:, off:off + s.shape[1] * 4] = s.view(torch.uint8)
        st["base"], st["stride"] = base, stride
        st["x"] = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
        st["counts"], st["offsets"], st["sorted_idx"] = _groups(T, E, k, g)
        st["cap"] = int(st["counts"].max())
        st["y"] = torch.zeros(T * k, H, dtype=torch.bfloat16, device=DEV)
    if own:
        moe = _package()
        if op == "balance":
            need = moe.moe_balance_loss_workspace(case["T"], case["E"], case["S"])
        elif op == "matmul":
            need = moe.moe_fp8_matmul_workspace(case["M"], case["N"], case["K"], max(case["E"], 1))
        elif op == "ffn":
            st["W"] = moe.experts("fp8_b128", case["E"], case["H"], case["I"], st["base"],
                                  st["stride"])
            need = moe.moe_expert_ffn_fp8_workspace(st["W"], case["T"], case["k"])
        else:
            need = 0
        st["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _valid(st):
    """(v, q): which tokens count, and each token's sequence (clamped)."""
    seq = st["seq"].to(torch.int64)
    T, S = st["logits"].shape[0], seq.numel() - 1
    t = torch.arange(T, device=DEV)
    q = torch.searchsorted(seq, t, right=True) - 1
    v = (q >= 0) & (q < S)
    if st["mask"] is not None:
        v = v & (st["mask"] != 0)
    return v, q.clamp(0, S - 1)


def _seq_sum(x, seq):
    """Sums of x's rows over each sequence (prefix sums in the type of x)."""
    c = torch.cat([torch.zeros_like(x[:1]), x.cumsum(0)])
    s = seq.to(torch.int64)
    return c[s[1:]] - c[s[:-1]]


def _counts(st, v, q):
    E, S = st["logits"].shape[1], st["seq"].numel() - 1
    key = q[:, None] * E + st["ids"].to(torch.int64)
    add = v[:, None].expand_as(key).to(torch.int32)
    flat = torch.zeros(S * E, dtype=torch.int32, device=DEV)
    return flat.scatter_add_(0, key.reshape(-1), add.reshape(-1)).view(S, E)


def _softmax(x):
    z = torch.exp(x - x.amax(1, keepdim=True))
    return z / z.sum(1, keepdim=True)


def _balance_plain(st):
    k, E = st["case"]["k"], st["case"]["E"]
    v, q = _valid(st)
    p = _softmax(st["logits"]) * v[:, None]
    probs = _seq_sum(p.double(), st["seq"])
    n = _seq_sum(v.to(torch.int64), st["seq"])
    counts = _counts(st, v, q)
    nd = n.double().clamp(min=1.0)
    loss = (counts * probs).sum(1) * (E / k) / (nd * nd)
    return n.to(torch.int32), counts, probs.float(), loss.float()


def _route_grad_plain(st):
    case = st["case"]
    k, E = case["k"], case["E"]
    v, q = _valid(st)
    p = _softmax(st["logits"])
    n = st["n"].float().clamp(min=1.0)
    a = st["dloss"] * (E / k) / (n * n)
    c = st["counts"].float() * a[:, None]
    ct = c[q]
    g = p * (ct - (p * ct).sum(1, keepdim=True))
    wd = st["w"] * st["dw"]
    tot = wd.sum(1, keepdim=True)
    ids = st["ids"].to(torch.int64)
    if case["renorm"]:
        g = g.scatter_add(1, ids, wd - st["w"] * tot)
    else:
        g = (g - p * tot).scatter_add(1, ids, wd)
    return torch.where(v[:, None], g, torch.zeros_like(g))


def _quantize(x):
    """Rows of a floating matrix -> (codes, scales) by the definition; x in 32 or 64 bits."""
    T, K = x.shape
    kb = _up(K, 128) // 128
    b = torch.nn.functional.pad(x, (0, kb * 128 - K)).view(T, kb, 128)
    amax = b.abs().amax(2)
    m, e = torch.frexp(amax)                       # amax = m 2^e, 1/2 <= m < 1
    s = torch.where(m <= 0.875, e - 9, e - 8)      # 448 = 0.875 * 2^9
    scale = torch.exp2(s.clamp(min=-126).to(x.dtype))
    scale = torch.where(amax > 0, scale, torch.ones_like(scale))
    codes = (b / scale[:, :, None]).to(torch.float8_e4m3fn)
    return codes.view(T, kb * 128)[:, :K].contiguous(), scale


def _scaled(codes, scales, dtype):
    """The values of E4M3 codes [..., R, K] with one scale per row and 128 columns."""
    K = codes.shape[-1]
    return codes.to(dtype) * scales.to(dtype).repeat_interleave(128, -1)[..., :K]


def _scaled_w(codes, scales, dtype):
    """The values of E4M3 codes [..., N, K] with one scale per 128 x 128 block."""
    N, K = codes.shape[-2:]
    s = scales.to(dtype).repeat_interleave(128, -1)[..., :K]
    return codes.to(dtype) * s.repeat_interleave(128, -2)[..., :N, :]


def _slots(offsets, counts, cap):
    """Row numbers [E, cap] of each expert's rows, and which of them exist."""
    i = torch.arange(cap, device=DEV)
    rows = offsets[:-1, None].to(torch.int64) + i
    return rows, i < counts[:, None]


def _grouped(a, w, st):
    """y[r] = a[r] w[e]^T for the rows r of each expert e, as one batched product."""
    rows, live = _slots(st["offsets"], st["counts"], st["cap"])
    y = torch.bmm(a[rows.clamp(max=a.shape[0] - 1)], w.transpose(1, 2))
    out = torch.zeros(a.shape[0], w.shape[1], device=DEV)
    out[rows[live]] = y[live]
    return out


def _matmul_plain(st):
    a = _scaled(st["a"], st["sa"], torch.float32)
    w = _scaled_w(st["w_"], st["sw"], torch.float32)
    y = _grouped(a, w, st) if st["case"]["E"] else a @ w.t()
    return y.to(torch.bfloat16)


def _record_parts(st):
    case = st["case"]
    E, H, I = case["E"], case["H"], case["I"]
    o13, o13s, o2, o2s, _ = _layout(H, I)
    b = st["base"]
    codes = lambda o, n, k: b[:, o:o + n * k].view(torch.float8_e4m3fn).view(E, n, k)  # noqa: E731
    scale = lambda o, n, k: (b[:, o:o + n * k // 128 // 128 * 4].contiguous()  # noqa: E731
                             .view(torch.float32).view(E, n // 128, k // 128))
    return codes(o13, 2 * I, H), scale(o13s, 2 * I, H), codes(o2, H, I), scale(o2s, H, I)


def _ffn_plain(st):
    I, k = st["case"]["I"], st["case"]["k"]
    w13, s13, w2, s2 = _record_parts(st)
    x = _scaled(*_quantize(st["x"].float()), torch.float32)
    rows = x[st["sorted_idx"].to(torch.int64) // k]
    gu = _grouped(rows, _scaled_w(w13, s13, torch.float32), st)
    gate, up = gu[:, :I], gu[:, I:]
    h = gate / (1.0 + torch.exp(-gate)) * up
    h = _scaled(*_quantize(h), torch.float32)
    return _grouped(h, _scaled_w(w2, s2, torch.float32), st).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own(st):
    moe = _package()
    case = st["case"]
    op = case["op"]
    if op == "balance":
        moe.moe_balance_loss(st["logits"], st["ids"], case["k"], st["n"], st["counts"], st["probs"],
                             st["loss"], st["ws"], token_mask=st["mask"], seq_offsets=st["seq"])
        return st["n"], st["counts"], st["probs"], st["loss"]
    if op == "route_grad":
        moe.moe_route_backward(st["logits"], case["k"], st["ids"], st["w"], st["dw"], st["n"],
                               st["counts"], st["dloss"], st["dlogits"], renorm=case["renorm"],
                               token_mask=st["mask"], seq_offsets=st["seq"])
        return st["dlogits"]
    if op == "quantize":
        moe.moe_fp8_quantize(st["x"], st["codes"], st["scales"])
        return st["codes"], st["scales"]
    if op == "matmul":
        moe.moe_fp8_matmul(st["a"], st["sa"], st["w_"], st["sw"], st["y"], st["ws"],
                           counts=st["counts"], offsets=st["offsets"])
        return st["y"]
    moe.moe_expert_ffn_fp8(st["W"], None, st["x"], case["T"], case["k"], st["counts"],
                           st["offsets"], st["sorted_idx"], st["y"], st["ws"])
    return st["y"]


_PLAIN = {"balance": _balance_plain, "route_grad": _route_grad_plain,
          "quantize": lambda st: _quantize(st["x"].float()), "matmul": _matmul_plain,
          "ffn": _ffn_plain}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# the same from the definitions in 64 bits
# ---------------------------------------------------------------------------
def _seq_lists(st):
    off = st["seq"].tolist()
    T = st["logits"].shape[0]
    ok = torch.ones(T, dtype=torch.bool, device=DEV) if st["mask"] is None else st["mask"].bool()
    return [torch.nonzero(ok[lo:hi]).flatten() + lo for lo, hi in zip(off[:-1], off[1:])]


def _e4m3(v):
    """Nearest-even E4M3 of 64-bit values within +-448, as 64-bit values."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 4).clamp(min=-9).double())   # 4 significant bits, 2^-9 at least
    return torch.round(v / step) * step


def _quantize_exact(x):
    T, K = x.shape
    vals, scales = torch.zeros_like(x), []
    for c in range(0, K, 128):
        b = x[:, c:c + 128]
        amax = b.abs().amax(1)
        s = torch.ceil(torch.log2(amax / QMAX)).clamp(-126, 200)
        s = torch.where(torch.exp2(s - 1) * QMAX >= amax, s - 1, s)   # log2 one too high
        s = torch.where(torch.exp2(s) * QMAX < amax, s + 1, s)        # or one too low
        s = torch.where(amax > 0, s.clamp(min=-126), torch.zeros_like(s))
        scales.append(torch.exp2(s))
        vals[:, c:c + 128] = _e4m3(b / torch.exp2(s)[:, None])
    return vals, torch.stack(scales, 1)


def _by_block(codes, scales, rows_too):
    v = codes.to(torch.float64)
    for c in range(0, v.shape[1], 128):
        s = scales[:, c // 128].double()
        v[:, c:c + 128] *= (s.repeat_interleave(128)[:v.shape[0]] if rows_too else s)[:, None]
    return v


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op in ("balance", "route_grad"):
        T, E, k = case["T"], case["E"], case["k"]
        x = st["logits"].double()
        p = torch.exp(x - torch.logsumexp(x, 1, keepdim=True))
        lists = _seq_lists(st)
        if op == "balance":
            probs = torch.stack([p[t].sum(0) for t in lists])
            counts = torch.stack([torch.bincount(st["ids"][t].flatten().long(), minlength=E)
                                  for t in lists])
            n = [max(len(t), 1) for t in lists]
            f = torch.tensor([E / (k * m * m) for m in n], dtype=torch.float64, device=DEV)
            return None, None, probs, (counts * probs).sum(1) * f
        out = torch.zeros(T, E, dtype=torch.float64, device=DEV)
        w, dw, ids = st["w"].double(), st["dw"].double(), st["ids"].long()
        for s, t in enumerate(lists):
            if not len(t):
                continue
            coef = float(st["dloss"][s]) * E / (k * len(t) ** 2)
            c = st["counts"][s].double() * coef
            pt = p[t]
            g = pt * (c - (pt @ c)[:, None])
            d = torch.zeros(len(t), E, dtype=torch.float64, device=DEV)
            inner = (w[t] * dw[t]).sum(1, keepdim=True)
            if case["renorm"]:
                d.scatter_(1, ids[t], w[t] * (dw[t] - inner))
            else:
                d.scatter_(1, ids[t], w[t] * dw[t])
                d -= pt * inner
            out[t] = g + d
        return out
    if op == "quantize":
        return _quantize_exact(st["x"].double())
    if op == "matmul":
        a = _by_block(st["a"], st["sa"], False)
        if not case["E"]:
            return a @ _by_block(st["w_"], st["sw"], True).t()
        y = torch.zeros(case["M"], case["N"], dtype=torch.float64, device=DEV)
        off = st["offsets"].tolist()
        for e in range(case["E"]):
            lo, hi = off[e], off[e + 1]
            if hi > lo:
                y[lo:hi] = a[lo:hi] @ _by_block(st["w_"][e], st["sw"][e], True).t()
        return y
    I, k = case["I"], case["k"]
    w13, s13, w2, s2 = _record_parts(st)
    v, s = _quantize_exact(st["x"].double())
    x = _by_block(v, s, False)
    off, tok = st["offsets"].tolist(), st["sorted_idx"].long() // k
    y = torch.zeros(case["T"] * k, case["H"], dtype=torch.float64, device=DEV)
    for e in range(case["E"]):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            gu = x[tok[lo:hi]] @ _by_block(w13[e], s13[e], True).t()
            h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
            hv, hs = _quantize_exact(h)
            y[lo:hi] = _by_block(hv, hs, False) @ _by_block(w2[e], s2[e], True).t()
    return y
