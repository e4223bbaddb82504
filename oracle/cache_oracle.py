"""Plain fp64 forms of the operators on a paged cache of keys and values (test
infrastructure; numpy only, nothing shared with the kernels).

Error bounds.  Attention: a score is an fp32 sum of D exact products, off by at
most D * 2^-24 of the sum of their magnitudes, times the scale (two more
roundings); a weight is the exponential of that difference (its error there, plus
4 * 2^-24 of the exponential itself), rounded to fp16 (2^-11; where it is
subnormal there, half a step of 2^-24, for a weight held 2^7 times as large relative to a
maximum that is at most the greatest: 2^-32 of the largest weight), the same number for the values and for the sum of
the weights; sums over n keys add n * 2^-24 at most; the result is rounded once
(2^-11, or 2^-25 among the subnormals).  Rotation: sine and cosine to 2^-23, four fp32
roundings, one to fp16.
"""
from __future__ import annotations

import numpy as np


def places(offsets, lengths, T):
    """(sequence, place) of each row, -1 for rows of no sequence."""
    seq, place = np.full(T, -1), np.full(T, -1)
    for b in range(len(lengths)):
        for i, t in enumerate(range(offsets[b], offsets[b + 1])):
            seq[t], place[t] = b, lengths[b] - (offsets[b + 1] - offsets[b]) + i
    return seq, place


def rotate(x, positions, inv_freq, interleaved, axes=None):
    """x [T, heads, D] -> (rotated, bound before rounding)."""
    x = x.astype(np.float64)
    y, e = x.copy(), np.zeros_like(x)
    R = 2 * len(inv_freq)
    for i, f in enumerate(inv_freq):
        p = positions if positions.ndim == 1 else positions[:, 0 if axes is None else axes[i]]
        angle = p.astype(np.float64) * np.float64(f)
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, R // 2 + i)
        y[:, :, a], y[:, :, b] = x[:, :, a] * c - x[:, :, b] * s, x[:, :, b] * c + x[:, :, a] * s
        e[:, :, a] = e[:, :, b] = 4 * 2.0 ** -23 * (np.abs(x[:, :, a]) + np.abs(x[:, :, b]))
    return y, e


def attend_row(q, k, v, scale):
    """q [D], k, v [n, D] (the keys that the row sees) -> (y, bound of the fp16 result)."""
    D = len(q)
    if len(k) == 0:
        return np.zeros(D), np.zeros(D)
    q, k, v = q.astype(np.float64), k.astype(np.float64), v.astype(np.float64)
    score = scale * (k @ q)
    off = scale * (D + 4) * 2.0 ** -24 * (np.abs(k) @ np.abs(q))
    w = np.exp(score - score.max())
    w /= w.sum()
    y = w @ v
    each = 2.0 ** -11 + 2 * (off.max() + (8 + len(k)) * 2.0 ** -24)
    small = 2.0 ** -32 * w.max()
    bound = each * (w @ np.abs(v) + np.abs(y)) + small * (np.abs(v).sum(0) + len(k) * np.abs(y))
    return y, bound + np.abs(y) * 2.0 ** -11 + 2.0 ** -25


def scores(q, bounds):
    """q [G, D], bounds [pages, 2, D] -> a score per page."""
    q = q.astype(np.float64)[None]
    lo, hi = (bounds.astype(np.float64)[:, None, i] for i in (0, 1))
    with np.errstate(invalid="ignore"):  # (the side that a channel does not use may be anything)
        return np.where(q == 0, 0.0, np.where(q > 0, q * hi, q * lo)).sum((1, 2))


def select(q, bounds, have, count, first, recent):
    """The pages, -1 past the last."""
    out = np.full(count, -1)
    if have <= count:
        out[:have] = np.arange(have)
        return out
    s = scores(q, bounds[first:have - recent])
    s = np.where(np.isnan(s), -np.inf, s)
    order = sorted(range(len(s)), key=lambda i: (-s[i], i))[:count - first - recent]
    out[:] = np.concatenate([np.arange(first), np.sort(np.array(order, int)) + first, np.arange(have - recent, have)])
    return out
