"""Drawing a token from a row of logits (TEST INFRASTRUCTURE, see the package
docstring): temperature, top-k, min-p and top-p, then the inverse CDF.

With w_i = exp((z_i - max z) / T) the vocabulary is ordered by (z descending,
index ascending).  top-k keeps the first k tokens, min-p those with w >=
min_p, top-p the shortest prefix of what is left that holds top_p of its
mass; at least one token stays.  The token is the first kept one in index
order whose running weight exceeds u times the kept weight.  T <= 0 is
greedy.  NaN counts as -inf; equal +inf logits share the row.
"""
import numpy as np


def kept(z, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Weights float64 [V] of one row, 0 where a token is not kept; all 0 if
    nothing may be drawn."""
    z = np.asarray(z, dtype=np.float64)
    z = np.where(np.isnan(z), -np.inf, z)
    V = z.shape[0]
    w = np.zeros(V)
    m = z.max()
    if m == -np.inf:
        return w
    order = np.lexsort((np.arange(V), -z))
    greedy = not temperature > 0
    with np.errstate(over="ignore", invalid="ignore"):
        x = np.where(z == m, 0.0, np.where((z == -np.inf) | (m == np.inf), -np.inf,
                                           (z - m) / (1.0 if greedy else temperature)))
    ws = np.exp(x)[order]
    n = V
    if greedy:
        n = 1
    elif top_k > 0:
        n = min(top_k, V)
    if min_p > 0:
        n = min(n, max(1, int(np.sum(ws >= min(min_p, 1.0)))))
    if top_p < 1:
        c = np.cumsum(ws[:n])
        before = np.concatenate([[0.0], c[:-1]])
        n = max(1, int(np.sum(before < max(top_p, 0.0) * c[-1])))
    w[order[:n]] = ws[:n]
    return w


def draw(w, u):
    """(token, log-probability) drawn from the weights; (-1, -inf) if they
    are all 0."""
    total = w.sum()
    if total == 0:
        return -1, -np.inf
    u = min(max(float(u), 0.0), 1.0) if u == u else 0.0
    hit = np.flatnonzero((np.cumsum(w) > u * total) & (w > 0))
    i = int(hit[0]) if hit.size else int(np.flatnonzero(w)[-1])
    return i, float(np.log(w[i]) - np.log(total))


def sample_row(z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    w = kept(z, temperature, top_k, top_p, min_p)
    return draw(w, u)
