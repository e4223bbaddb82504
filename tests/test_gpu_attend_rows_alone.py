"""Queries that are not finite stay with their rows: every other row is the same bits as without them."""
from __future__ import annotations

import numpy as np
import pytest

from tests import _gpu as G
from tests._cache import Batch

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("new,past,shared", [([1, 1, 1], [300, 20, 5000], 0), ([3, 2, 4], [700, 0, 90], 0),
                                             ([40, 30], [200, 3], 0), ([300, 1], [50, 40], 0), ([1] * 20, [30] * 20, 320),
                                             ([60, 40], [9, 70], 160)])
def test_queries_that_are_not_finite(new, past, shared, D):
    awq = G.lib()
    b = Batch(new, past, 8, 2, D, 16, shared=shared, seed=sum(new))
    cache, seqs = b.device()
    pages = torch.arange(b.width, dtype=torch.int32, device="cuda").expand(b.T, 2, b.width).contiguous()
    calls = [lambda q: awq.attend(q, cache, seqs, shared=shared), lambda q: awq.attend_pages(q, cache, seqs, pages)]
    q = G.dev_f16(b.q)
    for call in calls:
        plain = call(q).reshape(b.T, 8, D)
        for bad in (float("nan"), float("inf"), -float("inf")):
            odd = q.clone().reshape(b.T, 8, D)
            rows = {(0, 0), (b.T // 2, 5), (b.T - 1, 7), (b.T - 1, 2)}
            for t, h in rows:
                odd[t, h, 1] = bad
            y = call(odd.reshape(b.T, 8 * D)).reshape(b.T, 8, D)
            same = (y == plain).all(2).cpu().numpy()
            for t in range(b.T):
                for h in range(8):
                    if (t, h) not in rows:
                        assert same[t, h], (t, h, bad)
            for t, h in rows:
                if np.isnan(bad):
                    assert bool(torch.isnan(y[t, h]).all()), (t, h)
