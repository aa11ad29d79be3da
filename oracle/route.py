"""Softmax top-k routing with per-expert counts and the balance loss, and its
gradient, in float64, token by token.  Test infrastructure only."""

from __future__ import annotations

import numpy as np


def route(logits, top_k, normalize=True, mask=None):
    """Returns (idx [T, k] int, weights [T, k], counts [E], loss, n, p [T, E])."""
    x = np.asarray(logits, np.float64)
    t, e = x.shape
    idx = np.full((t, top_k), -1, np.int64)
    w = np.zeros((t, top_k))
    p = np.zeros((t, e))
    n = 0
    for i in range(t):
        if mask is not None and not mask[i]:
            continue
        row = x[i]
        if np.isnan(row).any() or np.isposinf(row).any() or np.isneginf(row).all():
            continue
        n += 1
        z = np.exp(row - row.max())
        p[i] = z / z.sum()
        order = sorted((j for j in range(e) if row[j] > -np.inf), key=lambda j: (-row[j], j))
        chosen = order[:top_k]
        idx[i, :len(chosen)] = chosen
        w[i, :len(chosen)] = p[i, chosen]
        if normalize:
            w[i] /= w[i].sum()
    counts = np.bincount(idx[idx >= 0], minlength=e)
    loss = e / (top_k * n * n) * float(counts @ p.sum(0)) if n else 0.0
    return idx, w, counts, loss, n, p


def route_backward(p, idx, weights, counts, n, dweights, dloss, normalize=True):
    """The gradient of the logits, through dp and the softmax's Jacobian."""
    t, e = p.shape
    k = idx.shape[1]
    out = np.zeros((t, e))
    for i in range(t):
        if idx[i, 0] < 0:
            continue
        dp = np.zeros(e) if dloss is None else dloss * e / (k * n * n) * counts.astype(float)
        sel = idx[i][idx[i] >= 0]
        if dweights is not None:
            dw = np.asarray(dweights[i], np.float64)[:len(sel)]
            if normalize:
                z = p[i, sel].sum()
                dp[sel] += dw / z - (dw @ p[i, sel]) / z ** 2
            else:
                dp[sel] += dw
        out[i] = p[i] * (dp - p[i] @ dp)
    return out
