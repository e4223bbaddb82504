"""Scores of up to 10^9, exact in fp32, that differ by a few units: a weight is of the difference, so they are as exact as those
of small scores, in waves and in row tiles, in one part and in many whose greatest scores differ."""
from __future__ import annotations

import numpy as np
import pytest

from tests import _gpu as G
from tests._cache import Batch

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("new,past", [(1, 700), (1, 20000), (3, 5000), (200, 1500)])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("power", [9, 10, 11, 20, 23, 24, 26, 28, 30])
def test_scores_far_from_zero(power, sign, new, past, D):
    """Each score is sign * 2^power plus 0 to 3 steps (of 1, or of what fp32 holds there), by blocks: the greatest score of a
    run of keys, and of a part, is now one and now another."""
    b = Batch([new], [past], 2, 1, D, 32, seed=power)
    n = past + new
    step = max(1.0, 2.0 ** (power - 23))
    at = np.arange(n)
    more = np.where(at < 40, 0, at // 96 % 4) * step * (at % 5 != 0)
    b.k[:] = 0
    half = power // 2
    page, slot = b.tables[0, at // 32], at % 32
    b.k[page, 0, slot, 0] = sign * 2.0 ** (power - half)
    b.k[page, 0, slot, 1] = more
    b.q[:] = 0
    q = b.q.reshape(b.T, 2, D)
    q[:, :, 0] = 2.0 ** half
    q[:, :, 1] = 1
    v = b.keys(0, 0, n, "v").astype(np.float64)
    cache, seqs = b.device()
    pages = torch.arange(b.width, dtype=torch.int32, device="cuda").expand(b.T, 1, b.width).contiguous()
    for y in (G.lib().attend(G.dev_f16(b.q), cache, seqs, scale=1.0), G.lib().attend(G.dev_f16(b.q), cache, seqs, scale=1.0, shared=448),
              G.lib().attend_pages(G.dev_f16(b.q), cache, seqs, pages, scale=1.0)):
        got = y.cpu().numpy().astype(np.float64).reshape(b.T, 2, D)
        for t in {0, new // 2, new - 1}:
            seen = past + t + 1
            w = np.exp(more[:seen] - more[:seen].max())
            w /= w.sum()
            ref, size = w @ v[:seen], w @ np.abs(v[:seen])
            # weights: to fp16 in numerator and denominator, 2^-11 of the values' size and of the result, and fp32: the
            # constant log2(e) and a part's greatest score times it (2^-24 of differences of at most 12, after the
            # maximum's own product is taken off exactly), exponentials and sums of `seen` numbers; the result's rounding
            each = 2.0 ** -11 + (32 + seen) * 2.0 ** -24
            bound = each * (size + np.abs(ref)) + np.abs(ref) * 2.0 ** -11 + 2.0 ** -25
            off = np.abs(got[t] - ref)
            assert np.all(off <= bound), (t, float((off / bound).max()))
