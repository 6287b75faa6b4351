"""Attention weights of cached tokens, and eviction by them, in float64.

Test infrastructure only (see ``oracle/__init__``).
"""

import numpy as np


def weights(q, lse, k, first, sm):
    """Weights [L] that the keys k [L, Hkv, d] get from rows q [n, Hq, d] with log-sum-exps lse [n, Hq], row i seeing
    positions 0 .. first + i, summed over rows and heads; and a bound on the sum's error in fp32.

    The bound: a score is an fp32 sum of d exact products (2^-24 of the sum of magnitudes for each of d terms and a
    few for the scale), and an f16 query element below 2^-14 is off by 2^-25; the exponent rounds once (2^-24 of it),
    the exponential and the row's factor are good to 2^-22 each, a weight below 2^-126 may be 0; the sum over N
    weights rounds N + 8 times."""
    n, hq, d = q.shape
    L, hkv = k.shape[:2]
    out, off = np.zeros(L), np.zeros(L)
    for h in range(hq):
        kh = k[:, h // (hq // hkv)]
        s = sm * q[:, h] @ kh.T
        with np.errstate(invalid="ignore"):
            x = s - lse[:, h, None]
        seen = np.arange(L)[None, :] <= first + np.arange(n)[:, None]
        seen &= ~np.isneginf(lse[:, h])[:, None]
        with np.errstate(invalid="ignore", over="ignore"):
            w = np.where(seen, np.exp(np.where(seen, x, 0.0)), 0.0)
            size = sm * np.abs(q[:, h]) @ np.abs(kh).T
            rel = (size * (d + 12) + np.abs(x)) * 2.0 ** -24 + sm * np.abs(kh).sum(1) * 2.0 ** -25 + 2.0 ** -21
            out += w.sum(0)
            off += np.where(seen, w * rel + 2.0 ** -126, 0.0).sum(0)
    return out, off + out * (n * hq + 8) * 2.0 ** -24


def keep(scores, budget, page=1, sinks=0, recent=0):
    """Which of a request's tokens stay (scores [n] fp32): True or False for each."""
    s = np.where(np.isnan(scores), -np.inf, scores)
    n = len(s)
    stays = np.ones(n, dtype=bool)
    if n <= budget:
        return stays
    pages = [list(range(a, min(a + page, n))) for a in range(0, n, page)]
    held = [p[0] < sinks or p[-1] >= n - recent or len(p) < page for p in pages]
    room = (max(budget, 0) - sum(len(p) for p, h in zip(pages, held) if h)) // page
    best = sorted((i for i, h in enumerate(held) if not h), key=lambda i: (-max(s[j] for j in pages[i]), i))
    for i in best[max(room, 0):]:
        stays[pages[i]] = False
    return stays
