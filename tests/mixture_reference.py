"""Plain 64-bit forms of the router, the grouping and the combination (numpy), from their definitions."""
from __future__ import annotations

import numpy as np

from rank_adapter_gemm_lora_amd import binding as lb


def route(x, top_k, score, renorm, scale):
    """(ids, weights, largest distance of a chosen logit from the row's maximum) of logits [rows, experts]."""
    rows, experts = x.shape
    ids = np.full((rows, top_k), -1, np.int32)
    w = np.zeros((rows, top_k))
    far = np.zeros(rows)
    for i in range(rows):
        on = [e for e in range(experts) if x[i, e] > -np.inf]     # neither -inf nor NaN
        chosen = sorted(on, key=lambda e: (-x[i, e], e))[:top_k]
        if not chosen:
            continue
        top = x[i, chosen[0]]
        if score == lb.LORA_MOE_SOFTMAX:
            def p(e):
                return 1.0 if x[i, e] == top else np.exp(x[i, e] - top)
            total = sum(p(e) for e in (chosen if renorm else on))
        else:
            low = min(top, 0.0) if renorm else 0.0

            def p(e):   # sigmoid(l), or that over exp(low)
                m = min(x[i, e], 0.0)
                return (1.0 if m == low else np.exp(m - low)) / (1 + np.exp(-abs(x[i, e])))
            total = sum(p(e) for e in chosen) if renorm else 1.0
        for j, e in enumerate(chosen):
            ids[i, j], w[i, j] = e, scale * p(e) / total
        finite = [x[i, e] for e in chosen if np.isfinite(x[i, e])]
        far[i] = max([abs(v) for v in finite] + [abs(v - top) for v in finite if np.isfinite(top)], default=0.0)
    return ids, w, far


def group(ids, experts):
    """(order, offsets, places) of ids [rows, top_k]."""
    key = np.where((ids < 0) | (ids >= experts), experts, ids).ravel()
    order = np.argsort(key, kind="stable").astype(np.int32)
    offsets = np.searchsorted(key[order], np.arange(experts + 1)).astype(np.int32)
    place = np.empty_like(order)
    place[order] = np.arange(len(order))
    return order, offsets, np.where(key < experts, place, -1)


def combine(y, place, w, residual):
    """(sum, sum of magnitudes) [rows, d] of y [pairs, d]."""
    rows, top_k = w.shape
    out = np.zeros((rows, y.shape[1])) if residual is None else residual.copy()
    size = np.abs(out)
    for j in range(top_k):
        at = place.reshape(rows, top_k)[:, j]
        on = at >= 0
        t = w[on, j, None] * y[at[on]]
        out[on] += t
        size[on] += np.abs(t)
    return out, size
