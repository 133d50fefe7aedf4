"""64-bit oracle of the routed experts' operators (test infrastructure only).

Plain numpy from the definitions.  Products come with the magnitude that a
rounding bound is stated against.
"""
from __future__ import annotations

import numpy as np

from . import q4k, q6k


def group(expert, experts, tokens=None):
    """(place, order, offsets) of the pairs with the experts ``expert``
    [tokens][top_k] (negative: none); tokens from ``tokens`` on lie behind the
    last."""
    expert = np.asarray(expert)
    flat = expert.reshape(-1)
    place, order, offsets = np.full(flat.size, -1, np.int32), np.full(flat.size, -1, np.int32), [0]
    for e in range(experts):
        mine = np.flatnonzero(flat == e)
        at = offsets[-1] + np.arange(len(mine))
        place[mine], order[at] = at, mine
        offsets.append(offsets[-1] + len(mine))
    place = place.reshape(expert.shape)
    if tokens is not None:
        place[tokens:] = -2
    return place, order, np.array(offsets, np.int32)


def route(logits, top_k, renormalize=True, scale=1.0, n_tokens=None):
    """(expert, weight, place, order, offsets)."""
    logits = np.asarray(logits, np.float64)
    tokens, experts = logits.shape
    live = tokens if n_tokens is None else min(max(n_tokens, 0), tokens)
    expert, weight = np.full((tokens, top_k), -1, np.int32), np.zeros((tokens, top_k))
    for t in range(live):
        have = [e for e in range(experts) if logits[t, e] > -np.inf]           # neither -inf nor NaN
        best = sorted(have, key=lambda e: (-logits[t, e], e))[:top_k]
        if not best:
            continue
        top = logits[t, best[0]]
        p = {e: 1.0 if logits[t, e] == top else float(np.exp(logits[t, e] - top)) for e in have}
        total = sum(p[e] for e in (best if renormalize else have))
        expert[t, :len(best)], weight[t, :len(best)] = best, [p[e] / total * scale for e in best]
    return (expert, weight, *group(expert, experts, live))


def _products(fields, fmt, rows, x):
    """x [n][cols] times the ``rows`` rows of ``fields``: (y, tolerance)."""
    if fmt == "q6_k":
        y, norm = q6k.gemv_q6k(fields, x)
        ones = q6k.gemv_q6k(fields, np.ones((1, x.shape[1]), np.float32))[1]
    else:
        y, norm = q4k.gemv(fields, x)[0], q4k.magnitude_norm(fields, x)
        ones = q4k.magnitude_norm(fields, np.ones((1, x.shape[1]), np.float32))
    return y, 1e-4 * (norm + 2.0 ** -16 * np.abs(x.astype(np.float64)).max(1, keepdims=True) * ones)


def _of(fields, e, rows):
    return {k: v[e * rows:(e + 1) * rows] for k, v in fields.items()}


def gate_up(x, gate, up, rows, expert, experts):
    """Rows of h in the order of the positions, and how far a result within
    the products' bounds may be from them."""
    _, order, offsets = group(expert, experts)
    n, top_k = offsets[-1], expert.shape[1]
    h, tol = np.zeros((n, rows)), np.zeros((n, rows))
    for e in range(experts):
        a, b = offsets[e], offsets[e + 1]
        if a == b:
            continue
        xs = np.asarray(x)[order[a:b] // top_k]
        (g, dg), (u, du) = (_products(_of(f, e, rows), "q4_k", rows, xs) for f in (gate, up))
        s = g / (1 + np.exp(-np.clip(g, -700, 700)))
        # |silu'| < 1.1; the function's own fp32 evaluation: a few half steps
        h[a:b], tol[a:b] = s * u, 1.1 * dg * (np.abs(u) + du) + np.abs(s) * du + 16 * 2.0 ** -24 * np.abs(s * u)
    return h, tol


def down(h, fields, fmt, rows, expert, weight, experts, residual=None):
    """(y, tolerance) [tokens][rows]."""
    place, _, offsets = group(expert, experts)
    y = np.zeros((len(expert), rows)) if residual is None else np.asarray(residual, np.float64).copy()
    tol = 1e-4 * np.abs(y)
    for e in range(experts):
        a, b = offsets[e], offsets[e + 1]
        if a == b:
            continue
        z, dz = _products(_of(fields, e, rows), fmt, rows, np.asarray(h)[a:b])
        for t, j in zip(*np.nonzero(expert == e)):
            w = float(weight[t, j])
            y[t] += w * z[place[t, j] - a]
            tol[t] += abs(w) * dz[place[t, j] - a]
    return y, tol
