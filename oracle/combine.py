"""Permuted rows -> token rows with the routing weights, and the gradients, in fp64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

``perm[t*top_k + j]`` is the row of slot ``j`` of token ``t``; an entry outside
``[0, num_rows)`` is a slot that is not routed here: it contributes nothing and
its weight gets the gradient 0.
"""
from __future__ import annotations

import numpy as np


def _slots(perm, num_rows, top_k):
    for s, p in enumerate(np.asarray(perm, dtype=np.int64).reshape(-1)):
        if 0 <= p < num_rows:
            yield s // top_k, s % top_k, p


def combine_rows(rows, perm, weights, T: int, top_k: int):
    """``(out, magnitude)``; ``weights`` None means ones."""
    rows = np.asarray(rows, dtype=np.float64)
    w = np.ones((T, top_k)) if weights is None else np.asarray(weights, dtype=np.float64)
    out, mag = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for t, j, p in _slots(perm, rows.shape[0], top_k):
        out[t] += w[t, j] * rows[p]
        mag[t] += np.abs(w[t, j] * rows[p])
    return out, mag


def combine_rows_backward(grad_out, rows, perm, weights):
    """``(grad_rows, grad_weights, magnitude of grad_weights, rows pointed at)``."""
    g, r = np.asarray(grad_out, np.float64), np.asarray(rows, np.float64)
    w = np.asarray(weights, dtype=np.float64)
    grad_rows, hit = np.zeros_like(r), np.zeros(r.shape[0], dtype=bool)
    grad_w, mag = np.zeros_like(w), np.zeros_like(w)
    for t, j, p in _slots(perm, r.shape[0], w.shape[1]):
        grad_rows[p] = w[t, j] * g[t]
        hit[p] = True
        grad_w[t, j] = r[p] @ g[t]
        mag[t, j] = np.abs(r[p] * g[t]).sum()
    return grad_rows, grad_w, mag, hit
