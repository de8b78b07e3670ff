"""Sampling by its definition in 64 bits (test helper): numpy, a row at a time.

A kernel's weights are off by some 2^-31 of themselves, so which token is drawn, or kept, is certain only where no sum
lies that near to its border.  ``draw`` returns None for the token where one does (tests draw few of those, and count them).
"""
import numpy as np

NEAR = 2.0 ** -28


def kept(x, temperature, top_k, top_p, min_p):
    """Indexes of the kept tokens in index order, their weights, and whether every border was clear."""
    x = np.asarray(x, dtype=np.float64)
    there = np.flatnonzero(x > -np.inf)
    if len(there) == 0:
        return there, np.zeros(0), True
    top = x[there].max()
    if top == np.inf:
        w = (x[there] == np.inf).astype(np.float64)
    else:
        with np.errstate(over="ignore"):
            w = np.exp((x[there] - top) / temperature)
    order = np.lexsort((there, -x[there]))
    at, w = there[order], w[order]
    w[w < 2.0 ** -44] = 0.0
    clear = True
    if top_k is not None and top_k > 0:
        at, w = at[:top_k], w[:top_k]
    if top_p is not None and top_p < 1:
        share = np.cumsum(w)
        want = max(top_p, 0.0) * share[-1]
        n = int(np.searchsorted(share, want)) + 1
        exact = len(np.unique(w[w > 0])) == 1  # equal weights: sums of ones, as exact there as here
        clear &= exact or np.abs(share - want).min() > NEAR * share[-1]
        at, w = at[:n], w[:n]
    if min_p is not None and min_p > 0:
        p = min(min_p, 1.0)
        clear &= p == 1.0 or np.abs(w - p).min() > NEAR
        at, w = at[w >= p], w[w >= p]
    back = np.argsort(at)
    return at[back], w[back], bool(clear)


def draw(x, u, temperature=1.0, top_k=None, top_p=None, min_p=None):
    """(token or None where a border is too near, confidence of the token)."""
    x = np.asarray(x, dtype=np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    top = x.max() if len(x) else -np.inf
    if top == -np.inf:
        return -1, 0.0
    if not temperature > 0:
        tok = int(np.flatnonzero(x == top)[0])
        clear = True
    else:
        at, w, clear = kept(x, temperature, top_k, top_p, min_p)
        share = np.cumsum(w)
        want = min(max(u, 0.0), 1.0) * share[-1]
        pick = int(np.searchsorted(share, want, side="right"))
        pick = min(pick, int(np.flatnonzero(w > 0)[-1]))
        tok = int(at[pick])
        exact = len(np.unique(w[w > 0])) == 1
        if not exact and u > 0 and u < 1:
            clear &= bool(np.abs(share - want).min() > NEAR * share[-1])
    soft = (x == np.inf).astype(np.float64) if top == np.inf else np.exp(x - top)
    return (tok if clear else None), float(soft[tok] / soft.sum())
