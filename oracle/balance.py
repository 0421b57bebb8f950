"""Load-balance loss of the router, and the gradients that reach its logits (oracle).

The pages describe serving and give no training formula.  Reading taken here
(stated with the ABI): per sequence s of a packed batch, with p = softmax of a
token's logits over the experts and only unmasked tokens counted,

  n_s = number of tokens, c_se = assignments to expert e, P_se = sum of p[t, e],
  loss_s = E / (k n_s^2) sum_e c_se P_se           (0 for n_s = 0),

the counts carrying no gradient.  A row of logits that are all -inf has p = 0.

Parity: pinned by the uniform router (loss 1), the collapsed router (loss E/k
times the probability mass on the chosen experts), central differences of the
loss and of the routing weights, and invariance to splitting a batch.
"""
from __future__ import annotations

import numpy as np


def softmax_rows(logits: np.ndarray) -> np.ndarray:
    x = np.asarray(logits, dtype=np.float64)
    m = x.max(axis=1, keepdims=True) if x.size else np.zeros((x.shape[0], 1))
    with np.errstate(invalid="ignore"):
        z = np.exp(x - np.where(np.isneginf(m), 0.0, m))
        s = z.sum(axis=1, keepdims=True)
        return z / np.where(s == 0.0, 1.0, s)


def _rows(T, token_mask, seq_offsets):
    off = np.asarray([0, T] if seq_offsets is None else seq_offsets, dtype=np.int64)
    ok = np.ones(T, bool) if token_mask is None else np.asarray(token_mask).astype(bool)
    return [np.arange(a, b)[ok[a:b]] for a, b in zip(off[:-1], off[1:])]


def balance_loss(logits, ids, k, token_mask=None, seq_offsets=None):
    """(n_tokens [S], counts [S,E], probs [S,E], loss [S]); probs and loss float64."""
    lg = np.asarray(logits)
    T, E = lg.shape
    rows = _rows(T, token_mask, seq_offsets)
    S = len(rows)
    n, counts = np.zeros(S, np.int64), np.zeros((S, E), np.int64)
    probs, loss = np.zeros((S, E)), np.zeros(S)
    for s, r in enumerate(rows):
        n[s] = len(r)
        if not len(r):
            continue
        i = np.asarray(ids).reshape(T, k)[r].ravel()
        counts[s] = np.bincount(i[(i >= 0) & (i < E)], minlength=E)
        probs[s] = softmax_rows(lg[r]).sum(axis=0)
        loss[s] = E / (k * len(r) ** 2) * np.dot(counts[s], probs[s])
    return n, counts, probs, loss


def route_backward(logits, k, renorm, ids, w, dw, n, counts, d_loss, d_before, token_mask=None,
                   seq_offsets=None):
    """(d_logits, magnitude): the gradient in float64 on a copy of d_before (rows of no sequence
    keep it), and per element the sum of the magnitudes of the terms it is made of."""
    lg = np.asarray(logits)
    T, E = lg.shape
    off = np.asarray([0, T] if seq_offsets is None else seq_offsets, dtype=np.int64)
    out = np.array(d_before, dtype=np.float64)
    mag = np.zeros((T, E))
    out[off[0]:off[-1]] = 0.0
    for s, r in enumerate(_rows(T, token_mask, seq_offsets)):
        for t in r:
            p = softmax_rows(lg[t:t + 1])[0]
            g, m = np.zeros(E), np.zeros(E)
            if d_loss is not None:
                c = float(d_loss[s]) * E / (k * float(n[s]) ** 2) * np.asarray(counts[s], float)
                g += p * (c - p @ c)
                m += p * (np.abs(c) + p @ np.abs(c))
            if dw is not None:
                i = np.asarray(ids).reshape(T, k)[t]
                keep = (i >= 0) & (i < E)
                wt = np.where(keep, np.asarray(w, np.float64).reshape(T, k)[t], 0.0)
                dt = np.where(keep, np.asarray(dw, np.float64).reshape(T, k)[t], 0.0)
                D, Da = wt @ dt, np.abs(wt) @ np.abs(dt)
                for j in range(k):
                    if keep[j]:
                        g[i[j]] += wt[j] * (dt[j] - (D if renorm else 0.0))
                        m[i[j]] += np.abs(wt[j]) * (np.abs(dt[j]) + Da)
                if not renorm:
                    g -= p * D
                    m += p * Da
            out[t], mag[t] = g, m
    return out, mag
