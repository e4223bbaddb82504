"""Shared keys with new tokens among them: each sees those up to its own place."""
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


def within(new, lengths, shared, Hq=8, Hkv=2, D=128, S=16, seed=0):
    """A batch whose sequences may be shorter than the shared keys, or have new tokens among them."""
    b = Batch(new, [max(0, n - shared - m) for m, n in zip(new, lengths)], Hq, Hkv, D, S, shared=shared, pad=1, seed=seed)
    for s, n in enumerate(lengths):
        b.lengths[s] = n
        b.place[b.offsets[s]:b.offsets[s + 1]] = n - new[s] + np.arange(new[s])
    return b


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("new,lengths,shared", [
    ([1, 1, 1], [65, 40, 64], 64),            # a sequence that ends within them, one at their last
    ([3, 1], [66, 70], 64),                   # new tokens on both sides of their end
    ([2, 5, 1], [1, 5, 100], 96),             # one with fewer tokens than rows
    ([100, 1], [100, 97], 96),                # a prompt that begins with them, beside a single token
    ([200, 33, 7], [200, 180, 161], 160),     # row tiles, and rows within them
    ([130], [130], 128),
])
def test_new_tokens_among_the_shared_keys(new, lengths, shared, D):
    """Each sees them up to its own place and no further."""
    b = within(new, lengths, shared, D=D, seed=len(new))
    y = attend(b)
    rows = [t for t in range(sum(new)) if t < 6 or t % 7 == 0 or b.seq[t] > 0]
    b.check(y, f"{new} new of {lengths}, {shared} shared, heads of {D}", rows=rows)


@pytest.mark.parametrize("new", [4, 150])
def test_shared_keys_that_are_not_finite_stay_unseen(new):
    """A key and a value at a place among the shared keys: rows before it see nothing of them."""
    b = within([new, 1], [new + 20, 200], 160)
    at = new // 2 + 20 if new + 20 < 160 else 100  # (a place that some of the new tokens are before)
    page, slot = b.tables[0, at // 16], at % 16
    b.k[page, :, slot, 3] = np.nan
    b.v[page, :, slot, ::5] = np.inf
    y = attend(b)
    before = [t for t in range(new) if b.place[t] < at]
    assert len(before) >= 2
    b.check(y, f"{new} new tokens, place {at}", rows=before)
    assert bool(torch.isnan(y[new]).any())  # (the other sequence sees it)
