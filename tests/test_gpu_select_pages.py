"""awq_select_pages against the definition: whole numbers equal; ties, scores that are not numbers, every count."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import cache_oracle as C
from tests import _gpu as G
from tests._cache import Batch

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def batch(new, past, Hq, Hkv, D, S, **kw):
    b = Batch(new, past, Hq, Hkv, D, S, **kw)
    b.bounds = np.sort(b.rng.standard_normal((b.k.shape[0], Hkv, 2, D)).astype(np.float16), axis=2)
    return b


def check(b, count, first=1, recent=1, rows=None):
    awq = G.lib()
    cache, seqs = b.device()
    cache = cache._replace(bounds=G.dev_f16(b.bounds))
    got = awq.select_pages(G.dev_f16(b.q), cache, seqs, count, first, recent).cpu().numpy()
    assert got.shape == (b.T, b.Hkv, count)
    width = b.Hq // b.Hkv * b.D
    for t in range(b.T) if rows is None else rows:
        if b.seq[t] < 0:
            continue
        have = int(b.place[t]) // b.S + 1
        for h in range(b.Hkv):
            q = b.q[t, h * width:(h + 1) * width].reshape(-1, b.D)
            ref = C.select(q, b.bounds[b.tables[b.seq[t], :have], h], have, count, first, recent)
            assert np.array_equal(got[t, h], ref), (t, h, have, count, first, recent)
    return got


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (8, 1), (14, 2), (64, 8), (40, 1)])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_heads(Hq, Hkv, D):
    check(batch([1, 2], [1500, 700], Hq, Hkv, D, 16, seed=Hq), 12)


@pytest.mark.parametrize("pages", [1, 2, 3, 15, 16, 17, 63, 64, 65, 66, 255, 256, 257, 300, 1100, 2500])
def test_page_counts(pages):
    b = batch([1], [16 * pages - 5], 4, 2, 64, 16, seed=pages)
    for count in {1, 2, 3, max(3, pages // 3), max(3, pages - 1), pages, pages + 1}:
        check(b, count, first=min(1, count - 1))


@pytest.mark.parametrize("count,first,recent", [(2, 1, 1), (2, 0, 1), (5, 0, 5), (5, 4, 1), (5, 2, 3), (30, 3, 4), (90, 0, 1)])
def test_first_and_recent(count, first, recent):
    check(batch([1, 1, 3], [1600, 16 * 89, 20], 8, 2, 128, 16, pad=1), count, first, recent)


@pytest.mark.parametrize("width", [512, 513])  # scores in one launch and in two
@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_wide_tables(D, width):
    for pages in (1, 3, 17, 64, 400, 512):
        b = batch([1, 2], [pages * 16 - 1, max(0, pages * 16 - 40)], 8, 2, D, 16, width=width, seed=pages)
        for count, first, recent in ((2, 1, 1), (9, 0, 1), (16, 3, 4), (6, 2, 4)):
            check(b, count, first, recent)
    b = batch([1], [500 * 16 - 1], 8, 1, D, 16, width=width)
    b.bounds[:] = 1.0  # all equal
    check(b, 50)
    b.bounds[::3] = 2.0
    check(b, 300)
    check(b, 150)
    b.bounds[::5, :, 0, 3] = np.nan
    b.bounds[::7, :, 1, 4] = np.inf
    check(b, 100)


def test_many_pages():
    check(batch([1], [16 * 9000], 8, 1, 64, 16), 128, 1, 2)
    check(batch([1], [16 * 20001], 2, 1, 64, 16), 5, 1, 2)


def test_ties_go_to_the_lower_page():
    b = batch([1, 1], [3000, 4100], 4, 2, 64, 16)
    b.bounds[:] = np.array([-1, 1], np.float16)[:, None]  # all pages alike
    check(b, 20)
    b.bounds[:] = np.sort(b.rng.integers(-1, 2, b.bounds.shape[:2] + (2, 1)), axis=2)  # a few kinds of page
    b.q[:] = b.rng.integers(-1, 2, b.q.shape)
    for count in (3, 20, 77, 150):
        check(b, count)
    b.q[:] = 0
    check(b, 20)


def test_scores_that_are_not_numbers():
    b = batch([1, 1, 1], [1600, 1600, 1600], 4, 2, 64, 16)
    b.bounds[b.rng.random(b.bounds.shape[0]) < 0.2] = np.nan
    b.bounds[b.rng.random(b.bounds.shape[0]) < 0.1, :, 1] = np.inf
    b.bounds[b.rng.random(b.bounds.shape[0]) < 0.1, :, 0] = -np.inf
    b.q[1] = np.nan
    check(b, 30)


def test_empty_sequences_and_rows_without_a_place():
    awq = G.lib()
    b = batch([2, 1], [0, 900], 8, 2, 128, 16)
    b.lengths[0] = 1
    b.place[:2] = [-1, 0]
    got = check(b, 7, rows=[1, 2])
    assert np.all(got[0] == -1) and awq is not None


def test_streams_and_graphs():
    awq = G.lib()
    b = batch([1, 2, 1], [3000, 1500, 40], 16, 2, 128, 16)
    cache, seqs = b.device()
    cache = cache._replace(bounds=G.dev_f16(b.bounds))
    q = G.dev_f16(b.q)
    eager = awq.select_pages(q, cache, seqs, 16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = awq.select_pages(q, cache, seqs, 16)
    for _ in range(4):
        out.zero_()
        graph.replay()
        awq.select_pages(q, cache, seqs, 4)
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def test_no_tokens_and_no_bounds():
    awq = G.lib()
    b = batch([1], [20], 8, 2, 128, 16)
    cache, seqs = b.device()
    q = G.dev_f16(b.q)
    with pytest.raises(ValueError):
        awq.select_pages(q, cache, seqs, 4)
    cache = cache._replace(bounds=G.dev_f16(b.bounds))
    assert awq.select_pages(q[:0], cache, seqs, 4).shape == (0, 2, 4)
