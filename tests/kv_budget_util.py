"""References of the attention weights and of what an eviction keeps, in float64 and plain
Python.  They share no code with the library."""

import numpy as np

import kv_util as U


def weights(q, k, ctx, count, scale, window, sinks):
    """Weights of one request: q [rows, heads, d], k [n, kv_heads, d], the first `count` rows.
    Returns (W [kv_heads, n], bound [kv_heads, n]).

    The bound: fp32 scores are off by at most (D + 8) 2^-24 of scale sum|q||k|, a weight by
    twice that in its exponent and twice in its divisor, a step of exp2 and of each sum over
    n terms; a step of each addition over the rows and heads; weights below 2^-126 may be 0."""
    rows, heads, d = q.shape
    n, kv = k.shape[:2]
    out, tol = np.zeros((kv, n)), np.zeros((kv, n))
    t = np.arange(n)
    for j in range(count):
        keep = U.sees(t, ctx + j, window, sinks)
        for h in range(heads):
            g = h // (heads // kv)
            with np.errstate(invalid="ignore", over="ignore"):
                s = scale * (k[keep, g] @ q[j, h])
                if not np.isfinite(s).all():
                    continue                              # such a row adds nothing
                w = np.exp(s - s.max())
            w = w / w.sum()
            slip = scale * (np.abs(k[keep, g]) @ np.abs(q[j, h])).max()
            out[g, keep] += w
            tol[g, keep] += w * (4 * (d + 8) * 2.0 ** -24 * slip + (2 * n + 128) * 2.0 ** -24
                                 + 2.0 ** -20) + 2.0 ** -126
    return out, tol + out * (count * (heads // kv) + 2) * 2.0 ** -24


def kept(w, n, m, sinks, recent):
    """Positions that stay of n, in order: the first, the last, and between them those of the
    largest weights (the lower position first among equals, NaN below everything)."""
    late = n - recent
    middle = sorted(range(sinks, late),
                    key=lambda t: (-np.inf if np.isnan(w[t]) else w[t], not np.isnan(w[t]), -t), reverse=True)
    return sorted(list(range(sinks)) + middle[:m - sinks - recent] + list(range(late, n)))


def evict_unit_bytes(units, page, d, keep):
    """What a request's units of one layer and KV head hold after an eviction: `units` [pages,
    unit] uint8 in the order of the table; the kept tokens' bytes move to the first slots, the
    other slots stay."""
    out = units.copy()
    places = U.places(page, d)
    for to, t in enumerate(keep):
        for at in places:
            out[to // page, at[to % page]] = units[t // page, at[t % page]]
    return out
