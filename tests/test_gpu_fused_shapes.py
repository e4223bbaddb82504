"""linear_fused refuses inputs whose last dimension is not the layer's, also where the number of elements would fit."""
from __future__ import annotations

import pytest

from tests import _fused as H
from tests import _gpu as G

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def halves(*shape):
    return torch.ones(shape, dtype=torch.float16, device="cuda")


def test_rows_of_another_width():
    awq = G.lib()
    pw, _ = H.packed_layer(awq, 64, 128, 32, True, 1)
    for x, y in ((halves(4, 2, 64), halves(4, 64)), (halves(2, 2, 256), halves(8, 64)), (halves(256), halves(2, 64)),
                 (halves(128, 3, 2), halves(6, 64)), (halves(4, 3, 50), None)):
        with pytest.raises(ValueError, match="x must"):
            awq.linear_fused(x, pw, y=y)
        if y is not None:
            assert bool((y == 1).all())


def test_residual_of_another_shape():
    awq = G.lib()
    pw, _ = H.packed_layer(awq, 64, 128, 32, True, 1)
    x = halves(2, 3, 128)
    for bad in (halves(2, 6, 32), halves(1, 3, 128), halves(6 * 64), halves(3, 2, 128)):
        with pytest.raises(ValueError, match="residual must"):
            awq.linear_fused(x, pw, residual=bad)
    want = awq.linear_fused(x, pw, residual=halves(2, 3, 64))
    assert torch.equal(awq.linear_fused(x, pw, residual=halves(6, 64)), want)
