"""A block's attention that is refused leaves the cache as it was."""
from __future__ import annotations

import numpy as np
import pytest

from tests import _gpu as G
from tests._fused import packed_layer

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def test_refused_calls_write_nothing():
    awq = G.lib()
    HQ, HKV, D, S, K, T = 8, 2, 64, 16, 256, 3
    pw, _ = packed_layer(awq, (HQ + 2 * HKV) * D, K, 128, True, 5)
    po, _ = packed_layer(awq, K, HQ * D, 64, False, 6)
    freq = torch.from_numpy((10000.0 ** (-np.arange(0, D, 2) / D)).astype(np.float32)).cuda()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    seqs = awq.Sequences(i32([0, 1, 3]), i32([40, 70]), torch.arange(12, dtype=torch.int32, device="cuda").reshape(2, 6))
    x = torch.randn((T, K), device="cuda").half()
    cache = awq.kv_cache(12, HKV, D, S)
    for t in cache:
        t.fill_(3.0)
    wide = torch.zeros((T, K + 12), dtype=torch.float16, device="cuda")
    no_bounds = cache._replace(bounds=None)
    for c, kw in ((no_bounds, dict(pages=3)), (cache, dict(pages=1)), (cache, dict(pages=3, recent=3)), (cache, dict(shared=8)),
                  (cache, dict(shared=16 * 7)), (cache, dict(shared=1 << 32)), (cache, dict(scale=0.0)),
                  (cache, dict(pages=3, scale=float("nan"))), (cache, dict(pages=1 << 27)),
                  (cache, dict(residual=wide[:, :K])), (cache, dict(residual=wide.flatten()[4:4 + T * K].reshape(T, K))),
                  (cache, dict(residual=x[:2])), (cache, dict(residual=x.cpu())), (cache, dict(residual=x.float())),
                  (cache._replace(bounds=cache.bounds.cpu()), dict(pages=3)),
                  (cache._replace(bounds=cache.bounds[:6]), dict(pages=3))):
        with pytest.raises((ValueError, awq.AwqError)):
            awq.attention(x, pw, po, c, seqs, freq, **kw)
        with pytest.raises((ValueError, awq.AwqError)):
            awq.attention(x, pw, pw, c, seqs, freq)  # an output layer of another width
        torch.cuda.synchronize()
        assert all(bool((t == 3.0).all()) for t in cache), kw
    for kw in (dict(pages=3), dict(shared=16), dict(residual=x), dict(scale=0.3, pages=5, first=0, recent=5)):
        for t in cache:
            t.fill_(3.0)
        y = awq.attention(x, pw, po, cache, seqs, freq, **kw)
        assert bool(torch.isfinite(y).all()) and not bool((cache.k == 3.0).all()), kw
