"""Plain references of the operators that cut rows of logits, in 64 bits on the
host, one row at a time. Nothing here shares code with the kernels."""
import math

import numpy as np

# Weights are held to 2^-33 of themselves (2^-26 from the exponent, the terms of
# the series, 2^-45 from the unit): sums of them are right to 2^-32, and what lies
# nearer to a border than this share of the sum may fall on either side.
NEAR = 2.0 ** -32


def cut_row(z, T, k, p, m):
    """(kept mask, weights, whether a border is too near to tell) of one row of
    float64 logits; None for a row or settings that cannot be used."""
    V = len(z)
    top = z.max() if not np.isnan(z).any() else math.nan
    if not math.isfinite(top) or not (T == 0 or 2.0 ** -64 <= T <= 2.0 ** 64) or k < 0 or not 0 <= p <= 1 or not 0 <= m <= 1:
        return None
    order = np.argsort(-z, kind="stable")
    with np.errstate(over="ignore"):
        w = np.exp((z - top) / (T or 1.0))
    ws = w[order]
    k = 1 if T == 0 else min(k or V, V)
    n, near = k, False
    if p < 1 and T != 0:
        total = np.cumsum(ws.astype(np.longdouble))
        goal = np.longdouble(p) * total[k - 1]
        n_p = int((total < goal).sum()) + 1
        n = min(n, n_p)
        if p > 0:
            gap = np.abs(total - goal) / total[k - 1]
            # sums of equal weights are whole numbers on both sides
            near = bool(((gap > 0) & (gap < NEAR)).any())
    if m > 0:
        n = min(n, int((ws >= m).sum()))
        near |= bool((np.abs(ws - m) < 1e-13 * m).any() and 0 < m < 1)
    keep = np.zeros(V, bool)
    keep[order[:max(n, 1)]] = True
    return keep, w, near


def draw(keep, w, u):
    """(token, its log-probability, whether u is too near an edge to tell)."""
    at = np.nonzero(keep)[0]
    total = np.cumsum(w[at].astype(np.longdouble))
    u = 0.0 if not u > 0 else min(float(u), 1.0)
    target = np.longdouble(u) * total[-1]
    j = int((total <= target).sum())
    if j == len(at):  # u of 1: the last that has any weight
        j = int(np.nonzero(w[at] > 2.0 ** -45)[0][-1])
    gap = np.abs(total - target) / total[-1]
    near = bool((gap[:-1] < NEAR).any()) if 0 < u < 1 else False
    return int(at[j]), math.log(w[at[j]]) - math.log(float(total[-1])) if w[at[j]] > 0 else -math.inf, near
