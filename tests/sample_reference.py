"""The sampler's definition (include/q8_decode.h) in numpy f64 and Python integers."""
from __future__ import annotations

import math

import numpy as np

UNIT = 1 << 44


def draw(logits, temperature, top_k, top_p, min_p, u):
    """(index, prob in f64) of one row; parameters as Python numbers, already f32 values."""
    l = np.asarray(logits, dtype=np.float32).astype(np.float64)
    cand = np.flatnonzero(l > -np.inf)
    if not len(cand):
        return -1, 0.0
    cand = cand[np.argsort(-l[cand], kind="stable")]
    v = l[cand]
    if not temperature > 0:
        return int(cand[0]), 1.0
    with np.errstate(invalid="ignore", over="ignore"):
        x = np.where(v == v[0], 0.0, (v - v[0]) * (1.0 / temperature if temperature < math.inf else 0.0))
    w = [int(t) for t in np.floor(np.exp(np.where(np.isnan(x), -np.inf, x)) * float(UNIT) + 0.5)]
    c, total = [], 0
    for t in w:
        total += t
        c.append(total)
    keep = len(w) if top_k <= 0 else min(top_k, len(w))
    n_k = keep
    if top_p < 1:
        keep = min(keep, 1 + sum(1 for t in c[:n_k] if float(t) < top_p * float(c[n_k - 1])))
    if min_p > 0:
        keep = max(1, min(keep, sum(1 for t in w if float(t) >= min_p * float(UNIT))))
    kept = c[keep - 1]
    for j in range(keep):
        if float(c[j]) > u * float(kept) or c[j] >= kept:
            return int(cand[j]), w[j] / kept
    raise AssertionError("unreachable")
