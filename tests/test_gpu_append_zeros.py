"""awq_append_kv: the sign of a page's bounds that are zero, and signalling NaN, do not depend on how many tokens come at once."""
from __future__ import annotations

import numpy as np
import pytest

from tests import _gpu as G
from tests._cache import Batch

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("rotary", [0, 64])
def test_zeros_and_signalling_nan_at_once_and_one_by_one(rotary):
    awq = G.lib()
    b = Batch([48], [0], 2, 1, 64, 16)
    _, seqs = b.device()
    bits = b.rng.choice(np.array([0x0000, 0x8000], np.uint16), (48, 4, 64))
    bits[:, :, 32:] = b.rng.choice(np.array([0x0000, 0x8000, 0x7C01, 0xFC01, 0x7E00, 0x3C00, 0xBC00], np.uint16), (48, 4, 32))
    x = torch.from_numpy(bits.reshape(48, 256).view(np.int16)).cuda().view(torch.float16)
    freq = torch.zeros(rotary // 2, dtype=torch.float32, device="cuda") if rotary else None
    caches = []
    for steps in ([48], [1] * 48, [5, 16, 1, 15, 11]):
        cache, _ = b.device()
        cache = cache._replace(bounds=torch.zeros((cache.k.shape[0], 1, 2, 64), dtype=torch.float16, device="cuda"))
        at = 0
        for n in steps:
            one = awq.Sequences(torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                                torch.tensor([at + n], dtype=torch.int32, device="cuda"), seqs.tables)
            awq.append_kv(x[at:at + n], cache, one, freq)
            at += n
        caches.append(cache)
    for cache in caches[1:]:
        for a, c in zip(caches[0], cache):
            assert torch.equal(a.view(torch.int16), c.view(torch.int16))
    used = caches[0].bounds[torch.from_numpy(b.tables[0, :3]).cuda()]
    assert not bool(torch.isnan(used).any())
