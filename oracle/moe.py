"""A mixture-of-experts layer in fp64 (test infrastructure only).

Readings: picks are the top_k largest logits, a NaN above every number, ties to
the lowest index; their weights are the softmax over all experts at the picks,
divided by the picks' sum when renormalised; an expert's rows are its gate rows,
then its up rows; a token's output is the sum over its picks among the experts
held, zero without any.
"""

from __future__ import annotations

import numpy as np


def route(logits, top_k, renormalize):
    """(ids int [T, top_k] in descending order, weights [T, top_k])."""
    T, E = logits.shape
    ids = np.zeros((T, top_k), int)
    w = np.zeros((T, top_k))
    for t in range(T):
        left = list(range(E))
        for j in range(top_k):
            best = left[0]
            for e in left[1:]:
                a, b = logits[t, e], logits[t, best]
                if not np.isnan(b) and (np.isnan(a) or a > b):
                    best = e
            left.remove(best)
            ids[t, j] = best
        with np.errstate(invalid="ignore", over="ignore"):
            p = np.exp(logits[t] - np.max(logits[t]))
            w[t] = p[ids[t]] / (p[ids[t]].sum() if renormalize else p.sum())
    return ids, w


def layer(x, router, gate_up, down, top_k, renormalize=True, first=0, ids=None):
    """x [T, D], router [E, D], gate_up [local, 2F, D], down [local, D, F] -> dict with the output and the
    intermediate values that an error bound needs.  ``ids``: take these picks (whose logits a sum in another
    precision may order otherwise where they nearly tie) instead of the exact order's."""
    logits = x @ router.T
    if ids is None:
        ids, w = route(logits, top_k, renormalize)
    else:
        p = np.exp(logits - logits.max(1, keepdims=True))
        w = np.take_along_axis(p, ids, 1)
        w = w / (w.sum(1, keepdims=True) if renormalize else p.sum(1, keepdims=True))
    out = np.zeros_like(x)
    parts = {}
    F = gate_up.shape[1] // 2
    for t in range(x.shape[0]):
        for j, e in enumerate(ids[t]):
            if not first <= e < first + gate_up.shape[0]:
                continue
            with np.errstate(invalid="ignore", over="ignore"):
                v = gate_up[e - first] @ x[t]
                g, u = v[:F], v[F:]
                h = g / (1 + np.exp(-g)) * u
                y = down[e - first] @ h
                out[t] += w[t, j] * y
            parts[t, j] = (g, u, h, y)
    return dict(out=out, ids=ids, weights=w, logits=logits, parts=parts)
