"""Inputs and checks shared by the tests of the fused layer and the expert products."""
from __future__ import annotations

import numpy as np

import workloads
from oracle import awq_oracle as O
from tests import _gpu as G


def packed_layer(awq, N, K, g, zp, seed):
    """A packed layer on the GPU and its decoded weight (fp64) from the oracle."""
    W = workloads.weight(N, K, cfg=11, layer=seed % 1000, row_offset=bool(seed & 1))
    qw, sc, qz = O.pack(W, g, zp)
    wdq = O.dequant_packed(qw, sc, qz, N, K, g, zp)
    return awq.PackedWeight(*G.upload_packed(qw, sc, qz), N, K, g, zp), wdq


def packed_experts(awq, E, N, K, g, zp, seed):
    """A stack of packed layers on the GPU and their decoded weights."""
    parts = [O.pack(workloads.weight(N, K, cfg=12, layer=(seed + e) % 1000), g, zp) for e in range(E)]
    wdq = [O.dequant_packed(*p, N, K, g, zp) for p in parts]
    qw, sc = np.stack([p[0] for p in parts]), np.stack([p[1] for p in parts])
    qz = np.stack([p[2] for p in parts]) if zp else None
    return awq.PackedExperts(*G.upload_packed(qw, sc, qz), E, N, K, g, zp), wdq


def halves(shape, seed, scale=1.0):
    return (np.random.default_rng([17, seed]).standard_normal(shape) * scale).astype(np.float16)


def check(y, ref, bound, what):
    """Every element within its bound, and the whole within 1e-3 in the 2-norm.

    The 2-norm: weight and output roundings are independent, each at most
    2^-11 / sqrt 3 = 2.8e-4 of what it rounds in the mean square; a gated product
    meets three of them (both factors' weights and the output, the gate's
    stretched by its slope), 2.8e-4 * sqrt(1 + 1 + 1.3 ** 2) = 5.4e-4: 1e-3 leaves
    a factor of two for short rows."""
    y = np.asarray(y, np.float64)
    assert y.shape == ref.shape, what
    assert np.all(np.isfinite(y)), f"{what}: non-finite output"
    worst = float(np.max(np.abs(y - ref) / bound)) if y.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.2f} times the bound"
    norm = float(np.linalg.norm(ref))
    off = float(np.linalg.norm(y - ref))
    assert off <= 1e-3 * norm + 2.0 ** -24 * np.sqrt(y.size), f"{what}: 2-norm error {off / max(norm, 1e-300):.2e}"
