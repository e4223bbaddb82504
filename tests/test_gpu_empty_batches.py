"""No tokens at all (a process whose share of a batch is empty): empty results of the right shapes, in every call."""
from __future__ import annotations

import pytest

from tests import _fused as H
from tests import _gpu as G

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def halves(*shape):
    return torch.zeros(shape, dtype=torch.float16, device="cuda")


def test_fused_layer_without_tokens():
    awq = G.lib()
    up, _ = H.packed_layer(awq, 64, 128, 32, True, 1)
    down, _ = H.packed_layer(awq, 128, 32, 32, True, 2)
    assert awq.linear_fused(halves(0, 128), up).shape == (0, 64)
    assert awq.linear_fused(halves(2, 0, 128), up, gated=True, residual=halves(2, 0, 32)).shape == (2, 0, 32)
    y = halves(0, 64)
    assert awq.linear_fused(halves(0, 128), up, halves(64), "silu", y=y) is y
    assert awq.mlp(halves(0, 128), up, down, residual=halves(0, 128)).shape == (0, 128)
    for bad in (halves(0, 64), halves(0, 128).float()):
        with pytest.raises(ValueError):
            awq.linear_fused(bad, up)
    with pytest.raises(ValueError, match="activation"):
        awq.linear_fused(halves(0, 128), up, activation="tanh")
    with pytest.raises(ValueError, match="residual"):
        awq.linear_fused(halves(0, 128), up, residual=halves(1, 64))


def test_experts_without_tokens():
    awq = G.lib()
    E, k = 6, 2
    up, _ = H.packed_experts(awq, E, 64, 128, 32, True, 1)
    down, _ = H.packed_experts(awq, E, 128, 32, 32, True, 2)
    for dtype in (torch.float16, torch.float32):
        route = awq.route_experts(torch.zeros((0, E), dtype=dtype, device="cuda"), k)
        assert [tuple(t.shape) for t in route] == [(0, k), (0, k), (E + 1,), (0,), (0, k)]
        assert [t.dtype for t in route] == [torch.int32, torch.float32, torch.int32, torch.int32, torch.int32]
        assert bool((route.offsets == 0).all())
    h = awq.linear_experts(halves(0, 128), up, route, activation="silu", gated=True)
    assert h.shape == (0, 32)
    assert awq.combine_experts(h, down, route, residual=halves(0, 128)).shape == (0, 128)
    assert awq.expert_mlp(halves(0, 128), halves(0, E), up, down, k, residual=halves(0, 128)).shape == (0, 128)
    with pytest.raises(awq.AwqError):
        awq.route_experts(halves(0, E), E + 1)
    with pytest.raises(ValueError):
        awq.linear_experts(halves(1, 128), up, route)
