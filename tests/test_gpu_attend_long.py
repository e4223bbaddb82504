"""Attention over tens of thousands of keys, whose parts many waves or splits make: every block of 32 keys counts, with its
own weight (tests/_cache_long.py)."""
from __future__ import annotations

import numpy as np
import pytest

from tests import _cache_long as L
from tests import _gpu as G
from tests._cache import Batch

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def put(b, which, s, h, rows):
    """The keys (values) of sequence s, key head h."""
    n, S = len(rows), b.S
    at = np.arange(n)
    getattr(b, which)[b.tables[s, at // S], h, at % S] = rows


def results(b, shared=0, **kw):
    """attend, with and without shared keys, and attend_pages over all pages, as [T, Hq, D]."""
    awq = G.lib()
    cache, seqs = b.device()
    q = G.dev_f16(b.q)
    out = [awq.attend(q, cache, seqs, shared=0, **kw)]
    if shared:
        out.append(awq.attend(q, cache, seqs, shared=shared, **kw))
    pages = torch.arange(b.width, dtype=torch.int32, device="cuda").expand(b.T, b.Hkv, b.width).contiguous()
    out.append(awq.attend_pages(q, cache, seqs, pages, **kw))
    return [y.cpu().numpy().reshape(b.T, b.Hq, b.D) for y in out]


CASES = [([1], [20011], 128), ([1], [65537], 128), ([1, 1], [20011, 65], 64), ([1], [20011], 96), ([1], [20011], 256),
         ([30], [20011], 128), ([30], [20011], 256)]


@pytest.mark.parametrize("new,past,D", CASES)
def test_the_whole(new, past, D):
    b = Batch(new, past, 8, 2, D, 32, seed=past[0])
    rows = [0, b.T - 1]
    ref = b.expected(rows=rows)[0].reshape(len(rows), 8, D)
    for y in results(b, shared=past[0] // 64 * 32 if len(new) == 1 else 0):
        L.check_norm(y[rows], ref, f"{new} after {past}, heads of {D}")


@pytest.mark.parametrize("new,past,D", CASES)
def test_every_block_counts(new, past, D):
    b = Batch(new, past, 8, 2, D, 32, seed=past[0])
    b.q[:] = 0
    kept = {}
    for s, n in enumerate(b.lengths):
        for h in range(2):
            kept[s, h] = np.roll(L.whole_values(n, D), h, 1)
            put(b, "v", s, h, kept[s, h])
    for y in results(b, shared=past[0] // 64 * 32 if len(new) == 1 else 0):
        for t in sorted({0, b.T // 2, b.T - 1}):
            for head in range(8):
                L.check_whole(y[t, head], kept[b.seq[t], head // 4][:b.place[t] + 1], f"row {t}, head {head}")


@pytest.mark.parametrize("new,past,D", [([1], [20011], 128), ([1], [65537], 64), ([1], [20011], 256), ([5], [20011], 96)])
def test_each_block_by_itself(new, past, D):
    """As many query heads as there may be for one key head, each looking for another block."""
    Hq = 256 if new == [1] else 64
    b = Batch(new, past, Hq, 1, D, 32, seed=past[0])
    n = past[0]  # (blocks that all rows see whole)
    put(b, "k", 0, 0, L.codes(np.arange(b.lengths[0]) // 32, D))
    v = b.keys(0, 0, b.lengths[0], "v")
    blocks = np.arange(n // 32)
    for first in range(0, len(blocks), Hq):
        here = blocks[first:first + Hq]
        q = np.zeros((Hq, D), np.float16)
        q[:len(here)] = L.codes(here, D)
        b.q[:] = q.reshape(1, -1)
        for y in results(b, shared=past[0] // 64 * 32, scale=L.CODE_SCALE):
            for t in range(b.T):
                for i, block in enumerate(here):
                    L.check_block(y[t, i], v, block, f"{new} after {past}, heads of {D}, row {t}")
