"""Gradients of the combine and of the expert FFN, rows into expert order and back, and
clipping by the global norm (oracle).

The pages describe serving and give no training formula.  These are the
derivatives of oracle.combine and oracle.ffn's definitions in float64, rows
p in expert order, row inv[a] for assignment a = t k + j of weight w[a]:

  dispatch:   x_perm[inv[a]] = w[a] x[t];  d_x[t] = sum_j w[a] d_x_perm[inv[a]],
              d_w[a] = <d_x_perm[inv[a]], x[t]>
  combine:    d_y_perm[inv[a]] = w[a] d_y[t];  d_w[a] = <y_perm[inv[a]], d_y[t]>
  FFN:        h = silu(g) u;  du = dh silu(g), dg = dh u silu'(g)
  clipping:   scale = min(1, max_norm / (norm + 1e-6))

An inv outside [0, R) is a dropped assignment (no row).

Parity: pinned by central differences of the layer's own forward, by the
adjoint identity <dispatch(x), r> = <x, dispatch_backward(r)>, and by a row's
gradient summed alone.
"""
from __future__ import annotations

import numpy as np


def _f(a):
    return np.asarray(a, dtype=np.float64)


def dispatch(x, inv, w, R):
    x = _f(x)
    T = x.shape[0]
    inv = np.asarray(inv).reshape(T, -1)
    out, named = np.zeros((R, x.shape[1])), np.zeros(R, bool)
    for t in range(T):
        for j, p in enumerate(inv[t]):
            if 0 <= p < R:
                out[p] = x[t] * (1.0 if w is None else float(np.asarray(w).reshape(inv.shape)[t, j]))
                named[p] = True
    return out, named


def _picked(rows, inv, T):
    """[T][k][H] rows of every assignment (zeros for dropped ones)."""
    rows = _f(rows)
    inv = np.asarray(inv).reshape(T, -1).astype(np.int64)
    ok = (inv >= 0) & (inv < rows.shape[0])
    out = np.zeros(inv.shape + (rows.shape[1],))
    out[ok] = rows[inv[ok]]
    return out


def dispatch_backward(d_x_perm, inv, w, x, add=None):
    x = _f(x)
    T = x.shape[0]
    r = _picked(d_x_perm, inv, T)
    wt = np.ones(r.shape[:2]) if w is None else _f(w).reshape(r.shape[:2])
    d_x = (wt[:, :, None] * r).sum(1) + (0.0 if add is None else _f(add))
    return d_x, (r * x[:, None, :]).sum(2)


def combine_backward(d_y, y_perm, inv, w):
    d_y = _f(d_y)
    T = d_y.shape[0]
    d_y_perm, _ = dispatch(d_y, inv, w, np.asarray(y_perm).shape[0])
    return d_y_perm, (_picked(y_perm, inv, T) * d_y[:, None, :]).sum(2)


def sigmoid(z):
    z = _f(z)
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0, e) / (1.0 + e)


def ffn_train(x_rows, offsets, w13, w2):
    """(gate_up, h, y) of rows in expert order."""
    x_rows = _f(x_rows)
    E, I = w2.shape[0], w2.shape[2]
    gu, h = np.zeros((len(x_rows), 2 * I)), np.zeros((len(x_rows), I))
    y = np.zeros((len(x_rows), w2.shape[1]))
    for e in range(E):
        p = slice(int(offsets[e]), int(offsets[e + 1]))
        gu[p] = x_rows[p] @ _f(w13[e]).T
        h[p] = gu[p, :I] * sigmoid(gu[p, :I]) * gu[p, I:]
        y[p] = h[p] @ _f(w2[e]).T
    return gu, h, y


def ffn_backward(x_rows, offsets, w13, w2, gate_up, d_y):
    """(d_x, d_w13, d_w2) from the kept gate and up products."""
    x_rows, gu, d_y = _f(x_rows), _f(gate_up), _f(d_y)
    E, H, I = w2.shape
    d_x, d_w13, d_w2 = np.zeros_like(x_rows), np.zeros((E, 2 * I, H)), np.zeros((E, H, I))
    for e in range(E):
        p = slice(int(offsets[e]), int(offsets[e + 1]))
        g, u = gu[p, :I], gu[p, I:]
        s = sigmoid(g)
        dh = d_y[p] @ _f(w2[e])
        dgu = np.concatenate([dh * u * s * (1.0 + g * (1.0 - s)), dh * g * s], axis=1)
        d_x[p] = dgu @ _f(w13[e])
        d_w13[e] = dgu.T @ x_rows[p]
        d_w2[e] = d_y[p].T @ (g * s * u)
    return d_x, d_w13, d_w2


def clip_grad_norm(grads, max_norm):
    """(norm, scale, clipped)."""
    norm = float(np.sqrt(sum(float((_f(g) ** 2).sum()) for g in grads)))
    scale = min(1.0, max_norm / (norm + 1e-6))
    return norm, scale, [_f(g) * scale for g in grads]
