"""The mixture-of-experts layer in 64 bits on the CPU, from the projection's oracle.

`experts` returns (Y, A): the f64 result and the error scale of each output,
A = sum over choices of gate * (sum of |block terms|) + |residual|, for the
gate of helpers.py.  The library rounds g, u and h to f32 as this does; every
other sum is f64 on both sides, and the output is rounded once.
"""
from __future__ import annotations

import numpy as np

import oracle


def _project(mode, blocks, n, k, x):
    rows = x.shape[0]
    if mode == "f32":
        return oracle.project(mode, blocks, n, k, rows, x=x)
    hi, lo, scale = oracle.quantize_act(mode, x)
    return oracle.project(mode, blocks, n, k, rows, hi=hi, lo=lo, scale=scale)


def route(x, router, top_k, renormalize=True):
    """(ids, gates in f64) of f32 x [rows][k] and router [experts][k]."""
    z = (x.astype(np.float64) @ router.astype(np.float64).T).astype(np.float32).astype(np.float64)
    ids = np.argsort(-z, axis=1, kind="stable")[:, :top_k]
    p = np.exp(z - z.max(axis=1, keepdims=True))
    chosen = np.take_along_axis(p, ids, 1)
    return ids.astype(np.int32), chosen / (chosen if renormalize else p).sum(axis=1, keepdims=True)


def hidden(g, u):
    g, u = g.astype(np.float32).astype(np.float64), u.astype(np.float32).astype(np.float64)
    return (g / (1.0 + np.exp(-g)) * u).astype(np.float32)


def experts(mode, w_gate, w_up, w_down, k, ff, x, ids, gates, residual=None):
    y = np.zeros(x.shape) if residual is None else residual.astype(np.float64)
    a = np.abs(y)
    for e in range(w_gate.shape[0]):
        rows = np.flatnonzero((ids == e).any(axis=1))
        if not len(rows):
            continue
        g, _ = _project(mode, w_gate[e], ff, k, x[rows])
        u, _ = _project(mode, w_up[e], ff, k, x[rows])
        d, da = _project(mode, w_down[e], k, ff, hidden(g, u))
        weight = np.where(ids[rows] == e, gates[rows].astype(np.float64), 0.0).sum(axis=1, keepdims=True)
        y[rows] += weight * d
        a[rows] += np.abs(weight) * da
    return y, a
