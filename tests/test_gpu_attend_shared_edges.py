"""Shared keys of a batch that begins with sequences without rows, whose tables hold anything."""
from __future__ import annotations

import numpy as np
import pytest

from tests import _gpu as G
from tests._cache import Batch

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def attend(b):
    cache, seqs = b.device()
    y = torch.full((b.T, b.Hq * b.D), 7.0, dtype=torch.float16, device="cuda")
    G.lib().attend(G.dev_f16(b.q), cache, seqs, shared=b.shared, y=y)
    assert bool((y[sum(b.new):] == 7.0).all()), "rows of no sequence were written"
    return y


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("new", [[0, 1, 1], [0, 0, 3, 0, 1], [0] * 63 + [1], [0] * 64 + [2, 1], [0] * 130 + [1, 0, 1],
                                 [0, 70, 90], [0] * 65 + [150, 1], [0, 0]])
def test_sequences_without_rows_come_first(new, D):
    """Of length 0, with tables of no page: the shared keys are read through the first table that has rows."""
    b = Batch(new, [(13 * i) % 40 for i in range(len(new))], 8, 2, D, 16, shared=160, pad=1, seed=len(new))
    for s, n in enumerate(new):
        if n > 0:
            break
        b.lengths[s] = 0
        b.tables[s] = np.array([-1, 1 << 30, 3, -(1 << 31)])[(s + np.arange(b.width)) % 4]
    y = attend(b)
    b.check(y, f"new tokens {new}, heads of {D}")
