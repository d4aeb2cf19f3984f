"""A projection with the low-rank adapters of many requests, and its gradients, in fp64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Row ``t`` has adapter ``ids[t]``; an id outside ``[0, L)`` is none.  Every function
returns its results with their magnitudes: the same sums over absolute values.
"""
from __future__ import annotations

import numpy as np


def _rows(ids, L):
    ids = np.asarray(ids, dtype=np.int64)
    return [(l, np.flatnonzero(ids == l)) for l in range(L)]


def mm_lora(x, w, a, b, ids, scale=None, bias=None):
    """``(out, |out|, act, |act|)``."""
    x, w, a, b = (np.asarray(t, dtype=np.float64) for t in (x, w, a, b))
    L, R = a.shape[:2]
    out, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        out, mag = out + np.asarray(bias, np.float64), mag + np.abs(np.asarray(bias, np.float64))
    act, amag = np.zeros((x.shape[0], R)), np.zeros((x.shape[0], R))
    for l, rows in _rows(ids, L):
        s = 1.0 if scale is None else float(scale[l])
        act[rows], amag[rows] = x[rows] @ a[l].T, np.abs(x[rows]) @ np.abs(a[l]).T
        out[rows] += s * (act[rows] @ b[l].T)
        mag[rows] += abs(s) * (amag[rows] @ np.abs(b[l]).T)
    return out, mag, act, amag


def mm_lora_backward(go, x, w, a, b, ids, scale=None):
    """``((gx, |gx|), (ga, |ga|), (gb, |gb|))``."""
    go, x, w, a, b = (np.asarray(t, dtype=np.float64) for t in (go, x, w, a, b))
    gx, mx = go @ w, np.abs(go) @ np.abs(w)
    ga, ma, gb, mb = np.zeros_like(a), np.zeros_like(a), np.zeros_like(b), np.zeros_like(b)
    for l, rows in _rows(ids, a.shape[0]):
        s = 1.0 if scale is None else float(scale[l])
        u, um = go[rows] @ b[l], np.abs(go[rows]) @ np.abs(b[l])
        v, vm = x[rows] @ a[l].T, np.abs(x[rows]) @ np.abs(a[l]).T
        gx[rows] += s * (u @ a[l])
        mx[rows] += abs(s) * (um @ np.abs(a[l]))
        ga[l], ma[l] = s * (u.T @ x[rows]), abs(s) * (um.T @ np.abs(x[rows]))
        gb[l], mb[l] = s * (go[rows].T @ v), abs(s) * (np.abs(go[rows]).T @ vm)
    return (gx, mx), (ga, ma), (gb, mb)
