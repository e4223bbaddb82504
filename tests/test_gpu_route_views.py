"""Router logits that are views: rows and columns of a larger matrix, at any element's address."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import fused_oracle as F
from tests import _gpu as G
from tests.test_gpu_route import logits_of

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("T,E", [(1, 60), (5, 9), (300, 60)])
def test_logits_at_any_address(T, E, dtype):
    awq = G.lib()
    v = logits_of(T + 3, E + 7, 31, dtype)
    whole = torch.from_numpy(v).cuda()
    for t0, e0 in ((1, 0), (0, 1), (2, 3), (3, 7)):
        ref = F.route(v[t0:t0 + T, e0:e0 + E], 4, True)
        got = awq.route_experts(whole[t0:t0 + T, e0:e0 + E], 4)
        for a, b in zip((got.ids, got.offsets, got.rows, got.positions), (ref[0], *ref[2:])):
            assert np.array_equal(a.cpu().numpy(), b), (t0, e0)
        # the bound of the router's weights: (2 + 64 + 10 + 1) 2^-24 at most
        assert np.all(np.abs(got.weights.cpu().numpy() - ref[1]) <= 80 * 2.0 ** -24 * ref[1]), (t0, e0)
