"""Linear layers whose rows choose their own weights (oracle).

Plain definitions in float64 and whole numbers, row by row: the plan of a
batch, a router's choice, the experts' products, the sum over a token's
experts, and low-rank adapters.  Nothing is sorted, blocked or batched beyond
one row's own product.
"""

import numpy as np

from . import int4, nvfp4


def plan(ids, groups):
    """(order, where, offsets) of choices: rows of group 0 in ascending order,
    then group 1's, ..., then the rows of no group."""
    ids = np.asarray(ids).ravel()
    runs = [[] for _ in range(groups + 1)]
    for row, g in enumerate(ids.tolist()):
        runs[g if 0 <= g < groups else groups].append(row)
    order = np.array([r for run in runs for r in run], dtype=np.int64)
    where = np.empty_like(order)
    where[order] = np.arange(order.size)
    return order, where, np.cumsum([0] + [len(r) for r in runs[:-1]])


def route(logits, top_k, renormalize):
    """(ids, weights) [tokens, top_k]: the largest logits, of equal ones the
    lowest expert, -1 where none is left; NaN and -infinity are not chosen."""
    logits = np.asarray(logits, dtype=np.float64)
    ids = np.full((logits.shape[0], top_k), -1)
    weights = np.zeros(ids.shape)
    for t, row in enumerate(logits):
        able = [e for e in range(row.size) if row[e] > -np.inf]
        chosen = sorted(able, key=lambda e: (-row[e], e))[:top_k]
        if not chosen:
            continue
        top = row[chosen[0]]
        term = {e: 1.0 if row[e] == top else np.exp(row[e] - top) for e in able}
        total = sum(term[e] for e in (chosen if renormalize else able))
        ids[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = [term[e] / total for e in chosen]
    return ids, weights


def silu(g):
    return g / (1.0 + np.exp(-g))


def weights_of(fmt, parts):
    """float64 weights [n, k] of an expert's canonical codes."""
    return int4.dequantize(*parts) if fmt == "int4" else nvfp4.dequantize(*parts)


def experts_product(x, weights, order, offsets, top_k, gather):
    """[pairs, n]: row p is x's row of place p times its expert's weights
    (float64 [n, k] each); zero where the pair has no expert."""
    out = np.zeros((order.size, weights[0].shape[0]))
    for e, w in enumerate(weights):
        for p in range(offsets[e], offsets[e + 1]):
            out[p] = w @ x[order[p] // top_k if gather else p]
    return out


def combine(rows, where, offsets, weights):
    """[tokens, n]: each token's weighted sum; pairs of no expert add nothing."""
    out = np.zeros((weights.shape[0], rows.shape[1]))
    for t in range(weights.shape[0]):
        for j in range(weights.shape[1]):
            p = where[t, j]
            if p < offsets[-1]:
                out[t] += weights[t, j] * rows[p]
    return out


def lora(y, x, a, b, scale, ids):
    """y + scale B (A x), row by row, and what bounds its error: (out, sums of
    |b| |u|, sums of |b| sums of |a| |x|, each times |scale|)."""
    out, mid, far = y.astype(np.float64).copy(), np.zeros(y.shape), np.zeros(y.shape)
    for t, i in enumerate(np.asarray(ids).tolist()):
        if 0 <= i < a.shape[0]:
            u = a[i] @ x[t]
            out[t] += scale[i] * (b[i] @ u)
            mid[t] = abs(scale[i]) * (np.abs(b[i]) @ np.abs(u))
            far[t] = abs(scale[i]) * (np.abs(b[i]) @ (np.abs(a[i]) @ np.abs(x[t])))
    return out, mid, far
