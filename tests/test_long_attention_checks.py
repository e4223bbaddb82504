"""The checks of attention over many keys (tests/_cache_long.py) take the exact result and reject it with 32 keys left out."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import cache_oracle as C
from tests import _cache_long as L


@pytest.mark.parametrize("n", [20012, 65538])
def test_a_block_left_out_is_rejected(n):
    rng = np.random.default_rng(n)
    D, blocks = 128, -(-n // 32)
    for block in (0, 1, blocks // 3, blocks - 2):
        kept = np.ones(n, bool)
        kept[32 * block:32 * block + 32] = False
        # the 2-norm, of standard normal inputs
        q, k, v = (rng.standard_normal(s).astype(np.float16) for s in ((D,), (n, D), (n, D)))
        y, _ = C.attend_row(q, k, v, D ** -0.5)
        L.check_norm(y.astype(np.float16), y, "exact")
        lost, _ = C.attend_row(q, k[kept], v[kept], D ** -0.5)
        with pytest.raises(AssertionError):
            L.check_norm(lost.astype(np.float16), y, "a block left out")
        # whole values: a block left out of the values' sums, or of both sums
        whole = L.whole_values(n, D).astype(np.float64)
        L.check_whole((whole.sum(0) / n).astype(np.float16), whole, "exact")
        for count in (n, n - 32):
            with pytest.raises(AssertionError):
                L.check_whole((whole[kept].sum(0) / count).astype(np.float16), whole, "a block left out")
        # one block with all the weight
        code = L.codes(np.arange(n) // 32, D)
        y, _ = C.attend_row(L.codes([block], D)[0], code, v, L.CODE_SCALE)
        L.check_block(y.astype(np.float16), v, block, "exact")
        lost, _ = C.attend_row(L.codes([block], D)[0], code[kept], v[kept], L.CODE_SCALE)
        with pytest.raises(AssertionError):
            L.check_block(lost.astype(np.float16), v, block, "left out")


def test_codes_tell_blocks_apart():
    blocks = np.arange(1 << L.BITS)
    code = L.codes(blocks, 64).astype(np.int32)
    product = code[:200] @ code.T
    assert np.all(product[np.arange(200), np.arange(200)] == 12)
    product[np.arange(200), np.arange(200)] = 0
    assert product.max() == 10
