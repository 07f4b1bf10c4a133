"""One token per row of logits: temperature, top-k, top-p, min-p and the draw
from a given number, in fp64.

The pages do not name sampling; the reading is the header's: tokens in order
(logit falling, id rising), top_k of them, of those the shortest beginning
whose weight reaches top_p of theirs, of those the ones whose weight is at
least min_p of the largest; the draw takes the lowest id whose kept weights up
to and with it exceed u times all kept weight.
"""
import numpy as np


def sample_row(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Returns (id, p, kept ids by order, margin): margin is how far, in parts of
    the largest weight, the nearest decision (top_p's border, min_p's border,
    the draw) is from going the other way; min_p's, which one weight decides and no
    sum of V of them, counts 8 V times (2^-45 of it like V 2^-42 of the others).
    (-1, 0, [], inf) without a token."""
    l = np.asarray(logits, dtype=np.float64)
    none = (-1, 0.0, np.zeros(0, dtype=np.int64), np.inf)
    if np.isnan(l).any() or np.any(l == np.inf) or not np.any(l > -np.inf):
        return none
    if not 0 <= u <= 1 or not temperature >= 0 or np.isnan(top_p) or not min_p <= 1:
        return none
    order = np.argsort(-l, kind="stable")
    order = order[l[order] > -np.inf]
    if temperature == 0:
        return int(order[0]), 1.0, order[:1], np.inf
    w = np.exp((l[order] - l[order[0]]) / temperature)
    margin = np.inf
    n = len(order) if top_k <= 0 else min(int(top_k), len(order))
    if top_p < 1:
        ends = np.cumsum(w[:n])
        before, want = ends - w[:n], top_p * ends[-1]
        margin = min(margin, np.abs(before[1:] - want).min(initial=np.inf))
        n = max(1, int(np.sum(before < want)))
    if min_p > 0:
        margin = min(margin, np.abs(w[1:n] - min_p).min(initial=np.inf) * 8 * len(l))
        n = int(np.sum(w[:n] >= min_p))
    kept = order[:n]
    by_id = np.argsort(kept)
    ends = np.cumsum(w[:n][by_id])
    aim = u * ends[-1]
    margin = min(margin, np.abs(ends[:-1] - aim).min(initial=np.inf), aim if aim > 0 else np.inf)
    at = min(int(np.sum(ends <= aim)), n - 1)
    return int(kept[by_id[at]]), float(w[:n][by_id[at]] / ends[-1]), kept, margin


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """Rows of logits; returns (ids, p, margins)."""
    rows = len(logits)

    def of(v, r, default):
        return default if v is None else v[r]

    got = [sample_row(logits[r], u[r], of(temperature, r, 1.0), of(top_k, r, 0), of(top_p, r, 1.0), of(min_p, r, 0.0))
           for r in range(rows)]
    return (np.array([g[0] for g in got]), np.array([g[1] for g in got]), np.array([g[3] for g in got]))
