"""Oracle of attention weights summed per cached token, and of eviction by
them, in numpy and 64 bits."""

from __future__ import annotations

import numpy as np

from . import kv_cache

__all__ = ["weights", "choose"]


def weights(q, codes, scale, low, n_q, window, softmax_scale, centre):
    """(sums, bound, seen) of one sequence: q [n_q, Hq, D]; keys' codes [n, H,
    D], scale and low [n, H].  sums [H, n]: softmax weights summed over the
    query rows that see a token.  bound: how far fp32 arithmetic may be off.
    seen [n]: tokens that some row sees.

    A logit is off by at most delta_j = 2^-18 |softmax_scale| (s_j sum_d |q_d|
    C_jd + L_j sum_d |q_d|): the products of query elements and codes are exact,
    up to 2 D / 16 fp32 accumulations and the scaling are off by 2^-23 of the
    magnitudes that they add each, whose sum is that, whether the kernel's codes
    count from 0 (c, with low_j) or from the middle (c - z, with low_j + z s_j):
    C_jd and L_j are the larger of the two.  And by 2^-21 of the row's largest
    logit (differences of rounded logits, maxima and logarithms of sums).  A
    weight p_j = e^x_j / sum_k e^x_k then by at most a factor e^(delta_j + ln
    sum_k p_k e^delta_k); exp2 adds 2^-21 of it, the fp32 sums of the row's
    tokens and of the token's rows 2^-24 each a term at most."""
    n, heads, d = codes.shape
    hq = q.shape[1]
    k = kv_cache.values(codes, scale, low)
    q = np.asarray(q, np.float64)
    sums, bound, seen = np.zeros((heads, n)), np.zeros((heads, n)), np.zeros(n, bool)
    s64, low64, c64 = (x.astype(np.float64) for x in (scale, low, codes))
    mid = np.maximum(np.abs(low64), np.abs(low64 + centre * s64))
    off, s64 = np.maximum(c64, np.abs(c64 - centre)), np.abs(s64)
    group = hq // heads
    for i in range(n_q):
        p = n - n_q + i
        lo = max(0, p - window + 1) if window else 0
        if p < 0:
            continue
        see = slice(lo, p + 1)
        seen[see] = True
        for h in range(hq):
            c = h // group
            x = softmax_scale * (k[see, c] @ q[i, h])
            aq = np.abs(q[i, h])
            delta = abs(softmax_scale) * 2.0 ** -18 * (s64[see, c] * (off[see, c] @ aq) + mid[see, c] * aq.sum())
            delta += 2.0 ** -21 * np.abs(x).max()
            w = np.exp(x - x.max())
            w /= w.sum()
            total = np.log((w * np.exp(delta)).sum())
            sums[c, see] += w
            bound[c, see] += w * np.expm1(delta + total)
    terms = n + n_q * group
    return sums, 1.01 * bound + (2.0 ** -21 + terms * 2.0 ** -24) * sums + terms * 1e-37, seen


def choose(w, n, budget, first, last):
    """Indices kept of n tokens with weights w [n], ascending."""
    if n <= budget:
        return np.arange(n)
    nan = np.isnan(w)
    w = np.where(nan, -np.inf, np.asarray(w, np.float64))
    middle = sorted(range(first, n - last), key=lambda j: (-w[j], nan[j], j))
    return np.array(sorted([*range(first), *middle[: budget - first - last], *range(n - last, n)]))
