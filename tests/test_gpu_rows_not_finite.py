"""Infinities and NaN in one row of x: all of that row's outputs show it, and no other row's do; in every kernel of the
fused layer, the expert products and the weighted sum."""
from __future__ import annotations

import numpy as np
import pytest

import workloads
from oracle import fused_oracle as F
from tests import _fused as H
from tests import _gpu as G
from tests.test_gpu_experts import device_route, logits_of

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def spoiled(X, rows):
    bad = X.copy()
    for i, r in enumerate(rows):
        bad[r, (37 * i + 5) % X.shape[1]] = (np.nan, np.inf, -np.inf)[i % 3]
    return bad


def check(y, ref, bound, rows, what):
    assert not np.isfinite(y[rows]).any(), f"{what}: a spoiled row has finite outputs"
    keep = np.setdiff1d(np.arange(len(y)), rows)
    H.check(y[keep], ref[keep], bound[keep], what)


@pytest.mark.parametrize("M,K,g", [(3, 288, 32), (8, 256, 64), (13, 11008, 128), (30, 288, 32), (100, 320, 64),
                                   (300, 288, 32), (600, 320, 64)])
def test_fused_layer(M, K, g, N=136):
    awq = G.lib()
    pw, wdq = H.packed_layer(awq, N, K, g, True, 6)
    X = workloads.activations(M, K, cfg=11, layer=6)
    rows = np.unique([1, M // 2, M - 1])
    y = G.host_f16(awq.linear_fused(G.dev_f16(spoiled(X, rows)), pw))
    check(y, *F.linear_fused(X, wdq), rows, f"M={M} K={K}")


@pytest.mark.parametrize("T,K,g", [(2, 256, 64), (7, 288, 32), (20, 288, 32), (20, 7168, 128), (100, 320, 64),
                                   (400, 288, 32), (700, 320, 64)])
def test_expert_layers(T, K, g, N=136):
    awq = G.lib()
    E, k = 8, 2
    ids, weights, offsets, rows, positions = F.route(logits_of(T, E, 61), k, True)
    route = device_route(awq, (ids, weights, offsets, rows, positions))
    pe, wdq = H.packed_experts(awq, E, N, K, g, True, 7)
    X = workloads.activations(T, K, cfg=12, layer=7)
    tokens = np.unique([0, T // 2])
    y = G.host_f16(awq.linear_experts(G.dev_f16(spoiled(X, tokens)), pe, route))
    check(y, *F.linear_experts(X, wdq, offsets, rows, k), np.flatnonzero(np.isin(rows // k, tokens)), f"rows T={T}")
    h, slots = workloads.activations(T * k, K, cfg=12, layer=8), np.unique([T // 3, T * k - 1])
    y = G.host_f16(awq.combine_experts(G.dev_f16(spoiled(h, slots)), pe, route))
    hit = np.flatnonzero(np.isin(positions, slots).any(1))
    check(y, *F.combine_experts(h, wdq, offsets, positions, weights.astype(np.float32)), hit, f"combined T={T}")


@pytest.mark.parametrize("M,N,K,g", [(700, 8200, 320, 64), (1100, 4104, 288, 32)])
def test_fused_layer_on_tiles(M, N, K, g):
    test_fused_layer(M, K, g, N)


@pytest.mark.parametrize("T,N,K,g", [(1500, 4104, 320, 64), (1500, 4104, 288, 32)])
def test_expert_layers_on_tiles(T, N, K, g):
    test_expert_layers(T, K, g, N)
