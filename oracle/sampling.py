"""CPU reference in float64 of the choice of the next token (test infrastructure): every row sorted, sum by sum."""

import numpy as np


def choose(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row: (token, log of its share, kept tokens, margin).  margin: how near, as a share of the sums compared, the
    row came to another result (borders of top_p, min_p and u)."""
    x = np.asarray(x, dtype=np.float64)
    ids = [i for i in range(len(x)) if x[i] > -np.inf]
    if not ids:
        return -1, -np.inf, 0, 1.0
    order = np.array(ids)[np.lexsort((ids, -x[ids]))]
    top = x[order[0]]
    margin = 1.0
    if not temperature > 0:
        return int(order[0]), 0.0, 1, margin
    if top == np.inf:
        order = order[x[order] == np.inf]
        w = np.ones(len(order))
    else:
        w = np.exp((x[order] - top) / temperature)
    n = len(order)
    if top_k > 0:
        n = min(n, int(top_k))
    if top_p < 1:
        total, run = w[:n].sum(), 0.0
        for i in range(n):
            run += w[i]
            margin = min(margin, abs(run - top_p * total) / total)
            if run >= top_p * total:
                n = i + 1
                break
    if min_p > 0:
        m = int((w[:n] >= min_p).sum())
        margin = min(margin, np.abs(w[1:n + 1] / min_p - 1).min() if len(w) > 1 else 1.0)
        n = max(1, min(n, m))
    c = np.cumsum(w[:n])
    u = min(u, 1 - 2.0 ** -52) if u > 0 else 0.0
    t = u * c[-1]
    if u > 0:
        margin = min(margin, np.abs(c[:-1] - t).min() / c[-1] if n > 1 else 1.0)
    at = min(int(np.searchsorted(c, t, side="right")), n - 1)
    return int(order[at]), float(np.log(w[at] / c[-1])), n, margin
