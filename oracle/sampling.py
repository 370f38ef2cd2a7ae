"""Temperature, top-k, top-p and min-p in fp64, and what a kept set and a drawn
token have to satisfy when weights carry a relative error.

Ranks are by (logit descending, id ascending) and -inf has none; every filter keeps a
prefix of the ranking.
"""

from __future__ import annotations

import numpy as np


def ranking(x):
    """ids of one row by rank, -inf left out."""
    x = np.asarray(x, np.float64)
    order = np.lexsort((np.arange(len(x)), -(x + 0.0)))
    return order[x[order] > -np.inf]


def weights(x, temperature):
    """(d, w) of one row; temperature 0: d undivided."""
    x = np.asarray(x, np.float64)
    d = (x - x.max()) / (temperature if temperature > 0 else 1.0)
    return d, np.exp(d)


def kept_bounds(x, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, tol=0.0):
    """(fewest, most) ranks that may be kept: borders within a relative tol of the sums
    or weights may go either way."""
    order = ranking(x)
    if len(order) == 0:
        return 0, 0
    _, w = weights(x, temperature)
    w = w[order]
    n = 1 if temperature <= 0 else min(top_k, len(order)) if top_k > 0 else len(order)
    w = w[:n]
    lo = hi = n
    if top_p < 1:
        before = np.cumsum(w) - w
        want = top_p * w.sum()
        lo, hi = [max(1, int((before < want * f).sum())) for f in (1 - tol, 1 + tol)]
    if min_p > 0:
        least = min(float(min_p), 1.0)
        lo = min(lo, max(1, int((w >= least * (1 + tol)).sum())))
        hi = min(hi, max(1, int((w >= least * (1 - tol)).sum())))
    return lo, hi


def draw_ok(x, kept_ids, token, u, temperature, tol):
    """Whether `token` may be drawn with u from the kept ids."""
    _, w = weights(x, temperature)
    ids = np.sort(kept_ids)
    cum = np.cumsum(w[ids])
    at = np.searchsorted(ids, token)
    if at >= len(ids) or ids[at] != token:
        return False
    want, slack = u * cum[-1], tol * cum[-1]
    return cum[at] > want - slack and cum[at] - w[token] <= want + slack
