"""Attention in 64 bits with a bound on what a kernel may differ by (test helper).

``attend`` computes o = sum_j w_j v_j, w = softmax(scale q k^T) over the seen
keys, for one query row, and the largest difference that the kernels' own
arithmetic can make:

* scores: a sum of ``head_dim`` products in fp32 is off by at most head_dim *
  2^-23 times the sum of their magnitudes (2^-24 a step, doubled for sums that
  are truncated instead of rounded); the scaling adds one rounding.  An error
  d of the exponents changes every weight by a factor within e^(+-d);
* the exponential: 2^-22 relative for ``ex2.approx`` plus one rounding of its
  argument, whose magnitude is at most the score range;
* the weights of the bf16 prompt kernel are rounded to bf16, 2^-8 relative each; the
  normaliser sums the rounded weights.  This is the default for bf16;
* so each weight is off by a factor 1 + r_j, |r_j| <= r, before normalising, and
  o by at most r sum_j w_j |v_j - o| / (1 - r);
* the bf16 token kernel holds a weight as two bf16: the first is cut off from the
  number just below it, the rest (at most 2^-7 of the weight's power of two) is rounded
  by half a step, 2^-9 of itself, so that 2^-16 of the weight is lost.  Its normaliser
  sums the weights as they were, so this moves o by at most 2^-16 sum_j w_j |v_j|
  (``weights`` = 2^-16, in place of the 2^-8 above);
* the fp32 sums over n keys: n 2^-23 sum_j w_j |v_j| at most, rescaling included;
* the output's own rounding: half a step of its type.
"""
import numpy as np


def attend(q, k, v, seen, scale, bf16, weights=None):
    """q [hd], k, v [n, hd] float64; seen [n] bool -> (o [hd], bound [hd])."""
    hd = q.shape[0]
    k, v = k[seen], v[seen]
    if len(k) == 0:
        return np.zeros(hd), np.zeros(hd)
    s = scale * (k @ q)
    w = np.exp(s - s.max())
    w /= w.sum()
    o = w @ v
    d = abs(scale) * (hd + 2) * 2.0 ** -23 * (np.abs(k) @ np.abs(q)).max()
    r = np.expm1(2 * d) + 2.0 ** -21 + (s.max() - s.min() + 8) * 2.0 ** -23
    if bf16 and weights is None:
        r = r + 2.0 ** -8 * (1 + r)
    spread = w @ np.abs(v - o)
    bound = r / (1 - r) * spread + ((len(k) + 64) * 2.0 ** -23 + (weights or 0.0) * (1 + r)) * (w @ np.abs(v))
    bound = bound + (2.0 ** -8 if bf16 else 2.0 ** -24) * (np.abs(o) + bound) + 1e-37
    return o, bound


def check(got, q, k, v, seen, scale, bf16, what="", weights=None):
    """Every row of got [rows, heads, hd] against attend(); k, v [keys, kv_heads, hd]; seen [rows, keys]."""
    got, q, k, v = (np.asarray(x, dtype=np.float64) for x in (got, q, k, v))
    group = q.shape[1] // k.shape[1]
    worst = 0.0
    for i in range(q.shape[0]):
        for h in range(q.shape[1]):
            o, tol = attend(q[i, h], k[:, h // group], v[:, h // group], seen[i], scale, bf16, weights)
            err = np.abs(got[i, h] - o)
            assert np.all(err <= tol), (what, i, h, float((err / tol).max()), got[i, h][:4], o[:4])
            worst = max(worst, float((err / np.maximum(tol, 1e-300)).max()))
    return worst


def window_mask(nq, nk, left, right, sinks):
    """seen [nq, nk] of row i at position nk - nq + i."""
    p = np.arange(nq)[:, None] + nk - nq
    j = np.arange(nk)[None, :]
    seen = np.ones((nq, nk), bool)
    if right >= 0:
        seen &= j <= p + right
    if left >= 0:
        seen &= (j >= p - left) | (j < sinks)
    return seen


def cancelling(rng, n, hd, heads, rounded):
    """q [heads, hd], k, v [n, hd] (values that `rounded` leaves as they are) whose outputs are sums that nearly cancel,
    column c for head c % heads: what is lost of a weight shows, as the output's own rounding is small.  Scores are single
    products, so that little is lost there."""
    k, q = np.zeros((n, hd)), np.zeros((heads, hd))
    k[:, 0] = rounded(-np.abs(rng.standard_normal(n)) * 2.0)
    q[:, 0] = rounded(1.0 + np.arange(heads) / 16.0)
    v = rounded(rng.standard_normal((n, hd)))
    at = rng.permutation(n)[:4]
    k[at, 0] = rounded(-rng.uniform(0.0, 0.5, 4))
    for c in range(hd):
        w = np.exp(q[c % heads, 0] * k[:, 0])
        w /= w.sum()
        v[at, c] = 0.0
        for j in at:  # each one takes what the others left, to its own rounding
            v[j, c] = rounded(-(w @ v[:, c]) / w[j])
    return q, k, v
