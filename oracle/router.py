"""The router of a MoE layer in fp64: top_k, counts, balance loss, gradients.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Plain loops over the tokens.
"""
from __future__ import annotations

import numpy as np


def softmax(z):
    """Of one row; -inf has probability 0, a row of -inf only has zeros."""
    z = np.asarray(z, dtype=np.float64)
    m = z.max()
    if m == -np.inf:
        return np.zeros_like(z)
    with np.errstate(invalid="ignore"):
        e = np.exp(z - m)
        return e / e.sum()


def topk(logits, k, renormalize=True, mask=None):
    """``(weights, ids)``: falling order, ties to the lowest index, -1 where nothing is left."""
    logits = np.asarray(logits, dtype=np.float64)
    T = logits.shape[0]
    w, ids = np.zeros((T, k)), np.full((T, k), -1, dtype=np.int32)
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        z, p = logits[t], softmax(logits[t])
        order = sorted((e for e in range(z.size) if z[e] != -np.inf),
                       key=lambda e: (0.0, e) if np.isnan(z[e]) else (1.0, -z[e], e))[:k]
        ids[t, : len(order)] = order
        w[t, : len(order)] = p[order]
        if renormalize and order:
            w[t] /= w[t].sum()
    return w, ids


def balance(logits, ids, coef, mask=None, given=None):
    """``(loss, counts, slopes)``."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    counts, mean, tokens = np.zeros(E, dtype=np.int64), np.zeros(E), 0
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        tokens += 1
        mean += softmax(logits[t])
        for e in ids[t]:
            if 0 <= e < E:
                counts[e] += 1
    by = counts if given is None else np.asarray(given, dtype=np.int64)
    if tokens == 0 or by.sum() == 0:
        return 0.0, counts, np.zeros(E)
    f = by / by.sum()
    return coef * E * float(f @ mean) / tokens, counts, coef * E * f / tokens


def backward(logits, k=1, ids=None, weights=None, grad_w=None, renormalize=True, slopes=None,
             grad_loss=0.0, mask=None):
    """Gradient of the logits, and the sum of its terms' absolute values."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        p = softmax(logits[t])
        q = np.zeros(E) if slopes is None else grad_loss * np.asarray(slopes, dtype=np.float64)
        q, qa = q.copy(), np.abs(q)
        if grad_w is not None:
            g, w = np.asarray(grad_w[t], np.float64), np.asarray(weights[t], np.float64)
            here = [j for j in range(k) if 0 <= ids[t, j] < E]
            c, ca = sum(g[j] * w[j] for j in here), sum(abs(g[j] * w[j]) for j in here)
            for j in here:
                e = ids[t, j]
                if renormalize:
                    out[t, e] += w[j] * (g[j] - c)
                    mag[t, e] += w[j] * (abs(g[j]) + ca)
                else:
                    q[e] += g[j]
                    qa[e] += abs(g[j])
        out[t] += p * (q - p @ q)
        mag[t] += p * (qa + p @ qa)
    return out, mag
