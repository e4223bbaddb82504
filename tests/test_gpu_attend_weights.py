"""The weights of attention, which the matrix cores take in 16 bits: small ones that count by their number, and results as
large as the values themselves, in row tiles (a prompt) and in waves (a single token), alone and with chosen pages."""
from __future__ import annotations

import numpy as np
import pytest

from tests import _gpu as G
from tests._cache import Batch

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def place(b, which, key, channel, value):
    """Channel `channel` of every key head's key (value) number `key` of the first sequence, or of all `key`s."""
    key = np.asarray(key)
    getattr(b, which)[b.tables[0, key // b.S], :, key % b.S, channel] = value


def attend(b, **kw):
    cache, seqs = b.device()
    return G.lib().attend(G.dev_f16(b.q), cache, seqs, **kw)


@pytest.mark.parametrize("power", [26, 30])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_small_weights_count(D, power):
    """One great key, all others 2^-power of it.  The bound is the oracle's: for 65536 keys at 2^-26 it is 2 % of what they
    give, and at 2^-30 a quarter."""
    n = 65536 if D == 64 else 32768
    b = Batch([n], [0], 1, 1, D, 64, width=n // 64)
    b.k[:] = 0
    b.v[:] = 0
    b.q[:] = 0
    b.q[:, 0] = 1
    keys = np.arange(n)
    place(b, "k", keys[1:], 0, -power * np.log(2.0))
    place(b, "v", keys[1:], 0, 1.0)   # what the small ones give
    place(b, "v", 0, 1, 1.0)          # what is left of the great one
    place(b, "v", keys[1::2], 2, -1.0)
    rows = [0, 1, 40, 5000, n // 2, n - 2, n - 1]
    b.check(attend(b, scale=1.0), f"{n} keys of 2^-{power}, heads of {D}", scale=1.0, rows=rows)


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("new", [1, 3, 200])
def test_results_as_large_as_the_largest_value(new, D):
    """All values of a channel the largest there is: an average cannot pass it, whichever way the weights are rounded.
    The weights, relative to the great keys' (one in 32), lie just above the middle between two halves, so that all are
    rounded up, or just below it, so that all are rounded down."""
    for side in (1.02, 0.98):
        b = Batch([new], [2000], 2, 1, D, 16)
        n = 2000 + new
        score = np.log(0.5 * (1 + side * 2.0 ** -11))
        high = np.float16(score)
        b.k[:] = 0
        b.q[:] = 0
        b.q.reshape(b.T, 2, D)[:, :, :2] = 1
        keys = np.arange(n)[np.arange(n) % 32 != 0]
        place(b, "k", keys, 0, high)
        place(b, "k", keys, 1, np.float16(score - np.float64(high)))
        place(b, "v", np.arange(n), 3, 65504.0)
        place(b, "v", np.arange(n), 4, -65504.0)
        results = [attend(b, scale=1.0)]
        cache, seqs = b.device()
        pages = torch.arange(b.width, dtype=torch.int32, device="cuda").expand(b.T, 1, b.width).contiguous()
        results.append(G.lib().attend_pages(G.dev_f16(b.q), cache, seqs, pages, scale=1.0))
        for y in results:
            y = y.reshape(b.T, 2, D).cpu().numpy()
            # (sums of 2000 products in fp32 are off by 2^-13 at most, 65504 is rounded to from 2^-12 above it)
            assert np.all(y[:, :, 3] == 65504.0) and np.all(y[:, :, 4] == -65504.0), (side, y[0, 0, 3:5])
            b.check(torch.from_numpy(y.reshape(b.T, 2 * D)), f"{new} rows, heads of {D}", scale=1.0)
