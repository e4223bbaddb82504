"""The paths that round no weight, held to it: every row of x has one channel that is not zero, so each output is one
product x (q - z) s, and the stored value is that product rounded once to fp16.  With weights rounded first many outputs
lie outside the bound."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import fused_oracle as F
from tests import _fused as H
from tests import _gpu as G
from tests.test_gpu_experts import device_route, logits_of

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

# x (q - z): 16 bits, exact; its product with the scale is rounded to 24 bits, and sums with zeros are exact.  Combining
# multiplies the scale by the slot's weight first, or the product by it, adds up to 4 terms and the residual.
ONE, COMBINED = 2.0 ** -23, 8 * 2.0 ** -24


def one_hot(rows, K, seed):
    rng = np.random.default_rng([23, rows, K, seed])
    X = np.zeros((rows, K), np.float16)
    X[np.arange(rows), rng.integers(0, K, rows)] = (rng.uniform(0.5, 2.0, rows) * rng.choice([-1, 1], rows))
    return X


def rounded_once(y, ref, rel, what):
    off = np.abs(y.astype(np.float64) - ref) / (np.abs(ref) * (2.0 ** -11 + rel) + 2.0 ** -25)
    assert np.max(off) <= 1.0, f"{what}: {np.max(off):.3f} times one rounding"


def test_bound_tells_rounded_weights():
    """The same bound on the oracle's values with weights rounded to fp16 first fails."""
    awq = G.lib()
    _, wdq = H.packed_layer(awq, 264, 512, 64, True, 3)
    X = one_hot(40, 512, 1).astype(np.float64)
    with pytest.raises(AssertionError):
        rounded_once((X @ wdq.astype(np.float16).astype(np.float64).T).astype(np.float16), X @ wdq.T, ONE, "rounded")
    rounded_once((X @ wdq.T).astype(np.float16), X @ wdq.T, ONE, "exact")


# up to 8 tokens with any groups, up to 256 with groups of 64 and more; K split in (13, 11008)
@pytest.mark.parametrize("M,K,g", [(1, 512, 32), (1, 512, 128), (2, 512, 32), (5, 1024, 64), (8, 512, 256), (9, 512, 64),
                                   (13, 11008, 128), (16, 512, 128), (33, 512, 64), (64, 4096, 256), (100, 1024, 128),
                                   (256, 512, 64)])
@pytest.mark.parametrize("zp", [True, False])
def test_fused_layer(M, K, g, zp):
    awq = G.lib()
    N = 264
    pw, wdq = H.packed_layer(awq, N, K, g, zp, M)
    X = one_hot(M, K, 2)
    rounded_once(G.host_f16(awq.linear_fused(G.dev_f16(X), pw)), X.astype(np.float64) @ wdq.T, ONE,
                 f"M={M} K={K} g={g} zp={zp}")


# up to 2 rows for each expert with any groups, up to 64 with groups of 64 and more
@pytest.mark.parametrize("T,K,g", [(1, 512, 32), (2, 512, 128), (7, 512, 32), (8, 1024, 64), (20, 512, 128),
                                   (20, 7168, 128), (100, 512, 64), (100, 2048, 128), (250, 512, 128)])
def test_expert_layers(T, K, g):
    awq = G.lib()
    E, N, k = 8, 136, 2
    ids, weights, offsets, rows, positions = F.route(logits_of(T, E, 51), k, True)
    route = device_route(awq, (ids, weights, offsets, rows, positions))
    pe, wdq = H.packed_experts(awq, E, N, K, g, True, T)
    X = one_hot(T, K, 3)
    expert = np.repeat(np.arange(E), np.diff(offsets))
    wide = [X[rows[r] // k].astype(np.float64) @ wdq[expert[r]].T for r in range(T * k)]
    rounded_once(G.host_f16(awq.linear_experts(G.dev_f16(X), pe, route)), np.stack(wide), ONE, f"rows T={T} K={K} g={g}")
    h, w32 = one_hot(T * k, K, 4), weights.astype(np.float32).astype(np.float64)
    terms = np.stack([h[r].astype(np.float64) @ wdq[expert[r]].T for r in range(T * k)])[positions] * w32[..., None]
    y = G.host_f16(awq.combine_experts(G.dev_f16(h), pe, route)).astype(np.float64)
    ref, size = terms.sum(1), np.abs(terms).sum(1)
    off = np.abs(y - ref) / (np.abs(ref) * 2.0 ** -11 + size * COMBINED + 2.0 ** -25)
    assert np.max(off) <= 1.0, f"combined T={T} K={K} g={g}: {np.max(off):.3f} times the bound"
