"""No batch size, group size or routing rounds a weight: outputs that are one product x (q - z) s, rounded once to fp16,
on the matrix-core tiles (several rounds, K split) and on the weight-stream tiles in groups of 32; and scales that are
zero, tiny and large side by side."""
from __future__ import annotations

import numpy as np
import pytest

import workloads
from oracle import awq_oracle as O
from oracle import fused_oracle as F
from tests import _fused as H
from tests import _gpu as G
from tests.test_gpu_exact_weights import one_hot, rounded_once
from tests.test_gpu_experts import device_route, logits_of

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def relative(K, g):
    """x (q - z) is exact.  The tiles carry a sum from multiples of one group's scale to multiples of the next: at most
    two roundings (the ratio, the product) for each group after the first, and the last scale's; sums with zeros are
    exact."""
    return (2 * (K // g) + 2) * 2.0 ** -24


@pytest.mark.parametrize("M,K,g", [(9, 512, 32), (13, 11008, 32), (40, 4096, 32), (100, 544, 32), (256, 512, 32),
                                   (257, 512, 32), (300, 544, 32), (300, 11008, 32), (300, 512, 64), (290, 4096, 64),
                                   (600, 320, 64), (300, 1024, 128), (400, 11008, 128), (300, 1024, 256)])
@pytest.mark.parametrize("zp", [True, False])
def test_fused_layer(M, K, g, zp, N=264):
    awq = G.lib()
    pw, wdq = H.packed_layer(awq, N, K, g, zp, M)
    X = one_hot(M, K, 2)
    ref = X.astype(np.float64) @ wdq.T
    rounded_once(G.host_f16(awq.linear_fused(G.dev_f16(X), pw)), ref, relative(K, g), f"M={M} K={K} g={g} zp={zp}")


# matrix-core tiles, one round of them and several; K split in (700, 4104)
@pytest.mark.parametrize("M,N,K,g", [(1100, 4104, 544, 32), (700, 8200, 512, 64), (700, 8200, 1024, 128),
                                     (700, 8200, 1024, 256), (700, 4104, 11008, 128)])
@pytest.mark.parametrize("zp", [True, False])
def test_fused_layer_on_tiles(M, N, K, g, zp):
    test_fused_layer(M, K, g, zp, N)


@pytest.mark.parametrize("E,T,K,g", [(8, 20, 512, 32), (8, 100, 544, 32), (8, 250, 512, 32), (8, 400, 544, 32),
                                     (8, 400, 512, 64), (4, 400, 4096, 128), (70, 2500, 256, 64), (70, 2500, 288, 32)])
def test_expert_layers(E, T, K, g, N=136):
    awq = G.lib()
    k = 2
    ids, weights, offsets, rows, positions = F.route(logits_of(T, E, 51), k, True)
    route = device_route(awq, (ids, weights, offsets, rows, positions))
    pe, wdq = H.packed_experts(awq, E, N, K, g, True, T)
    X = one_hot(T, K, 3)
    expert = np.repeat(np.arange(E), np.diff(offsets))
    flat = np.stack(wdq)

    def products(V):
        """Row r of V through its expert's weight: one term each."""
        at = np.argmax(V != 0, axis=1)
        return V[np.arange(len(V)), at].astype(np.float64)[:, None] * flat[expert, :, at]

    y = G.host_f16(awq.linear_experts(G.dev_f16(X), pe, route))
    rounded_once(y, products(X[rows // k]), relative(K, g), f"rows E={E} T={T} K={K} g={g}")
    h, w32 = one_hot(T * k, K, 4), weights.astype(np.float32).astype(np.float64)
    terms = products(h)[positions] * w32[..., None]
    y = G.host_f16(awq.combine_experts(G.dev_f16(h), pe, route)).astype(np.float64)
    ref, size = terms.sum(1), np.abs(terms).sum(1)
    bound = np.abs(ref) * 2.0 ** -11 + size * (relative(K, g) + 8 * 2.0 ** -24) + 2.0 ** -25
    assert np.max(np.abs(y - ref) / bound) <= 1.0, f"combined E={E} T={T} K={K} g={g}"


@pytest.mark.parametrize("E,T,N,K,g", [(8, 1500, 4104, 288, 32), (8, 1500, 4104, 320, 64), (70, 2500, 520, 288, 32),
                                       (8, 1000, 2056, 4096, 128)])
def test_expert_layers_on_tiles(E, T, N, K, g):
    test_expert_layers(E, T, K, g, N)


@pytest.mark.parametrize("M", [1, 5, 13, 40, 100, 300])
@pytest.mark.parametrize("K,g", [(544, 32), (512, 64), (1024, 128), (1024, 256)])
@pytest.mark.parametrize("zp", [True, False])
def test_scales_of_every_size(M, K, g, zp, N=136):
    """Groups whose scale is 0 (the first, the last, runs of them, whole rows), the smallest fp16 number, or 10^5 times
    it, next to each other, and negative ones."""
    awq = G.lib()
    Gr = K // g
    rng = np.random.default_rng([29, K, g, zp])
    qw, _, qz = O.pack(workloads.weight(N, K, cfg=11, layer=3), g, zp)
    s = rng.choice(np.array([0.0, 0.0, 2.0 ** -24, 3e-6, 1e-4, 0.02, -0.01]), (N, Gr))
    s[0::8, 0], s[1::8, -1], s[2::8], s[3::8, : Gr // 2], s[4::8, Gr // 2:] = 0.0, 0.0, 0.0, 0.0, 0.0
    s[5::8, 0::2], s[5::8, 1::2] = 2.0 ** -24, 0.02
    bits = s.astype(np.float16).reshape(N // 8, 8, Gr).transpose(0, 2, 1).copy().view(np.uint16)
    wdq = O.dequant_packed(qw, bits, qz, N, K, g, zp)
    assert np.count_nonzero(wdq[2]) == 0 and np.count_nonzero(wdq[5]) > 0
    pw = awq.PackedWeight(*G.upload_packed(qw, bits, qz), N, K, g, zp)
    X = workloads.activations(M, K, cfg=11, layer=M)
    y = G.host_f16(awq.linear_fused(G.dev_f16(X), pw))
    ref, bound = F.linear_fused(X, wdq)
    assert np.all(y[:, 2::8] == 0)
    H.check(y, ref, bound, f"M={M} K={K} g={g} zp={zp}")


@pytest.mark.parametrize("M,N,K,g", [(1100, 4104, 544, 32), (700, 8200, 512, 64), (700, 8200, 1024, 128),
                                     (700, 8200, 1024, 256)])
def test_scales_of_every_size_on_tiles(M, N, K, g):
    test_scales_of_every_size(M, K, g, g != 128, N)
