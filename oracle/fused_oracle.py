"""Plain fp64 forms of the fused layer, the expert router and the expert
products (test infrastructure; numpy only, nothing shared with the kernels).

Error bounds.  A kernel's sum differs from the exact one by at most
1e-3 * sum_k |x_k w'_k| (the layer's accuracy contract: one fp16 rounding per
weight, 2^-11, and fp32 accumulation); call that d.  An activation's slope is
at most 1.13 (silu: 1.10, gelu: 1.13), so act(v) is off by at most 1.13 d; a
gated product by 1.13 d_g |u| + |act(g)| d_u + 1.13 d_g d_u; a weighted sum by
the weighted sum of its terms' bounds.  The fp32 arithmetic of the epilogue
adds a few 2^-24 of each term (8 of them are allowed), and the stored fp16
value 2^-11 of the result, or 2^-25 among the subnormals.
"""
from __future__ import annotations

import math

import numpy as np

SUM_TOL = 1e-3
SLOPE = 1.13
EPS32 = 8 * 2.0 ** -24

_erf = np.vectorize(math.erf, otypes=[np.float64])


def activation(v: np.ndarray, name: str) -> np.ndarray:
    if name == "none":
        return v
    if name == "relu":
        return np.where(v < 0, 0.0, v)
    if name == "silu":
        return v / (1.0 + np.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1.0 + _erf(v / math.sqrt(2.0)))
    if name == "gelu_tanh":
        return 0.5 * v * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    raise ValueError(name)


def rounding(y: np.ndarray) -> np.ndarray:
    """The bound of one rounding to fp16."""
    return np.abs(y) * 2.0 ** -11 + 2.0 ** -25


def _product(X, Wdq, bias):
    """Exact pre-activations and the bound on the kernel's."""
    X, W = X.astype(np.float64), Wdq.astype(np.float64)
    v, d = X @ W.T, SUM_TOL * (np.abs(X) @ np.abs(W).T)
    if bias is not None:
        v = v + bias.astype(np.float64)
    return v, d + EPS32 * np.abs(v)


def epilogue_rows(X, Wdq, bias=None, act="none", gated=False):
    """fp64 rows and the bound on a kernel's unrounded ones."""
    v, d = _product(X, Wdq, bias)
    if gated:
        F = v.shape[1] // 2
        a, da = activation(v[:, :F], act), SLOPE * d[:, :F]
        u, du = v[:, F:], d[:, F:]
        y, e = a * u, da * np.abs(u) + np.abs(a) * du + da * du
    else:
        y, e = activation(v, act), SLOPE * d
    return y, e + EPS32 * np.abs(y)


def linear_fused(X, Wdq, bias=None, act="none", gated=False, residual=None):
    """(y, bound) of the fused layer's fp16 output."""
    y, e = epilogue_rows(X, Wdq, bias, act, gated)
    if residual is not None:
        r = residual.astype(np.float64)
        e = e + EPS32 * (np.abs(y) + np.abs(r))
        y = y + r
    return y, e + rounding(y)


def route(logits, top_k: int, renormalize: bool):
    """(ids, weights, offsets, rows, positions) by the definition, a token at a time."""
    T, E = logits.shape
    ids = np.full((T, top_k), -1, np.int32)
    weights = np.zeros((T, top_k), np.float64)
    for t in range(T):
        row = [float(v) for v in logits[t]]
        open_ = [e for e in range(E) if not math.isnan(row[e]) and row[e] != -math.inf]
        order = sorted(open_, key=lambda e: (-row[e], e))[:top_k]
        if not order:
            continue
        m = row[order[0]]
        share = lambda e: 1.0 if row[e] == m else math.exp(row[e] - m)  # noqa: E731
        total = math.fsum(share(e) for e in (order if renormalize else open_))
        for j, e in enumerate(order):
            ids[t, j] = e
            weights[t, j] = share(e) / total
    flat = ids.reshape(-1)
    slots = [s for e in range(E) for s in np.flatnonzero(flat == e)]
    offsets = np.concatenate([[0], np.cumsum([np.sum(flat == e) for e in range(E)])]).astype(np.int32)
    rows = np.full(T * top_k, -1, np.int32)
    rows[:len(slots)] = slots
    positions = np.full(T * top_k, -1, np.int32)
    positions[slots] = np.arange(len(slots), dtype=np.int32)
    return ids, weights, offsets, rows, positions.reshape(T, top_k)


def linear_experts(X, Wdq, offsets, rows, top_k, bias=None, act="none", gated=False):
    """(y, bound) of the routed rows, sorted by expert."""
    ys, es = [], []
    for e in range(len(Wdq)):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            y, d = epilogue_rows(X[rows[lo:hi] // top_k], Wdq[e], None if bias is None else bias[e], act, gated)
            ys.append(y)
            es.append(d + rounding(y))
    width = Wdq[0].shape[0] // (2 if gated else 1)
    return (np.concatenate(ys), np.concatenate(es)) if ys else (np.zeros((0, width)), np.zeros((0, width)))


def combine_experts(H, Wdq, offsets, positions, weights, bias=None, residual=None):
    """(y, bound) of each token's weighted sum over its slots."""
    T, top_k = positions.shape
    N = Wdq[0].shape[0]
    rows, bounds = np.zeros((H.shape[0], N)), np.zeros((H.shape[0], N))
    for e in range(len(Wdq)):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            rows[lo:hi], bounds[lo:hi] = _product(H[lo:hi], Wdq[e], None if bias is None else bias[e])
    y, d = np.zeros((T, N)), np.zeros((T, N))
    for t in range(T):
        for j in range(top_k):
            if positions[t, j] >= 0:
                w, r = float(weights[t, j]), positions[t, j]
                y[t] += w * rows[r]
                d[t] += w * bounds[r] + EPS32 * np.abs(w * rows[r])
    if residual is not None:
        d = d + EPS32 * (np.abs(y) + np.abs(residual.astype(np.float64)))
        y = y + residual.astype(np.float64)
    return y, d + rounding(y)
