"""Log probabilities of tokens, entropies and most probable tokens, in fp64.

For a row x: lse = ln(sum exp(x)), logprob of t = x[t] - lse, entropy =
-sum p ln p with 0 ln 0 = 0, alternatives by (logit descending, id
ascending).  A row of only -inf has no distribution: logprobs -inf, entropy 0.
A NaN or +inf in a row makes its numbers NaN (NaN ranks first among the ids).
"""

from __future__ import annotations

import numpy as np


def row_logprobs(x, token, k):
    """(logprob, entropy, top ids [k], top logprobs [k]) of one row."""
    x = np.asarray(x, dtype=np.float64)
    V = len(x)
    rank = np.where(np.isnan(x), np.inf, x + 0.0)
    order = np.lexsort((np.arange(V), -rank, ~np.isnan(x)))[:k]
    if np.isnan(x).any() or np.isposinf(x).any():
        return np.nan if 0 <= token < V else -np.inf, np.nan, order.astype(np.int32), np.full(k, np.nan)
    if np.isneginf(x).all():
        return -np.inf, 0.0, order.astype(np.int32), np.full(k, -np.inf)
    m = x.max()
    with np.errstate(all="ignore"):
        d = x - m
        e = np.exp(d)
        logs = np.log(e.sum())
        lp = d - logs
        p = np.exp(lp)
        entropy = -(p * np.where(p > 0, lp, 0.0)).sum()
    return lp[token] if 0 <= token < V else -np.inf, entropy, order.astype(np.int32), lp[order]


def emitted_tokens(tokens, path, accept_len, bonus, err):
    """[(b, k, row node, token)] of what each sequence emits."""
    out = []
    for b in range(len(bonus)):
        if err is not None and err[b] != 0:
            continue
        A = int(accept_len[b])
        for k in range(A + 1):
            token = int(tokens[b, path[b, k + 1] - 1]) if k < A else int(bonus[b])
            out.append((b, k, int(path[b, k]) - 1, token))
    return out
