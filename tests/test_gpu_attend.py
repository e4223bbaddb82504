"""awq_attend and awq_attend_pages against fp64 attention, row by row: head layouts, head sizes, page sizes, lengths from
none to long, ragged batches, shared prefixes, many new tokens, NaN and infinities wherever a row must not look."""
from __future__ import annotations

import numpy as np
import pytest

from tests import _gpu as G
from tests._cache import Batch

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

HEADS = [(1, 1), (4, 4), (8, 1), (10, 2), (14, 2), (16, 1), (36, 1), (40, 1), (64, 8)]


def attend(b, **kw):
    awq = G.lib()
    cache, seqs = b.device()
    y = torch.full((b.T, b.Hq * b.D), 7.0, dtype=torch.float16, device="cuda")
    awq.attend(G.dev_f16(b.q), cache, seqs, shared=b.shared, y=y, **kw)
    assert bool((y[sum(b.new):] == 7.0).all()), "rows of no sequence were written"
    return y


@pytest.mark.parametrize("Hq,Hkv", HEADS)
@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_heads(Hq, Hkv, D):
    b = Batch([1, 1, 1], [0, 70, 333], Hq, Hkv, D, 16, seed=Hq)
    b.check(attend(b), f"{Hq}/{Hkv} heads of {D}")


@pytest.mark.parametrize("S", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_page_sizes(S, D):
    b = Batch([1, 2, 1, 1], [S - 1, S - 2, 3 * S, 2 * S + 5], 8, 2, D, S, pad=2, seed=S)
    b.check(attend(b), f"pages of {S}, heads of {D}")


@pytest.mark.parametrize("past", [0, 1, 14, 15, 16, 17, 30, 31, 32, 33, 62, 63, 64, 65, 127, 128, 129, 1000])
def test_lengths(past):
    b = Batch([1], [past], 8, 1, 128, 16, seed=past)
    b.check(attend(b), f"{past} tokens before")


@pytest.mark.parametrize("past", [5000, 20011, 65537])
def test_long(past):
    b = Batch([1, 1], [past, 9], 8, 2, 128, 32, seed=past)
    b.check(attend(b), f"{past} tokens before")


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("new", [[2], [3, 1], [5, 2, 7], [31, 33], [64, 1, 65], [200]])
def test_several_new_tokens(new, D):
    b = Batch(new, [11 * i for i in range(len(new))], 8, 2, D, 16, pad=1, seed=len(new))
    b.check(attend(b), f"{new} new tokens, heads of {D}")


@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 1), (14, 2), (64, 8)])
def test_prompts(Hq, Hkv):
    b = Batch([300, 129, 1, 517], [0, 40, 700, 1000], Hq, Hkv, 128, 32, pad=3, seed=Hq)
    b.check(attend(b), f"prompts, {Hq}/{Hkv} heads")


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 4, 64), (8, 1, 128), (14, 2, 96), (64, 8, 128), (16, 1, 256)])
@pytest.mark.parametrize("B,new", [(1, 1), (2, 1), (13, 1), (40, 1), (5, 9)])
def test_shared(Hq, Hkv, D, B, new):
    b = Batch([new] * B, [(7 * i) % 50 for i in range(B)], Hq, Hkv, D, 16, shared=16 * 21, pad=1, seed=B)
    b.check(attend(b), f"{B} sequences after a shared prefix, {Hq}/{Hkv} heads of {D}")


@pytest.mark.parametrize("shared", [32, 64, 96, 2048, 6400])
def test_shared_lengths(shared):
    b = Batch([1, 4, 2], [0, 3, 90], 8, 2, 128, 32, shared=shared, seed=shared)
    b.check(attend(b), f"{shared} shared")


def test_shared_gives_what_separate_tables_give():
    b = Batch([1, 3, 1, 40], [0, 31, 7, 64], 8, 2, 128, 32, shared=640)
    y = attend(b)
    b.shared = 0
    z = attend(b)
    # (each is within its bound of the exact value: together within twice the larger part, weights rounded to fp16)
    assert float((y.float() - z.float()).abs().max()) <= 2.0 ** -9 * float(z.float().abs().max())


def test_a_row_without_keys_is_zero():
    awq = G.lib()
    b = Batch([1, 1, 1], [40, 3, 20], 8, 2, 128, 16)
    cache, seqs = b.device()
    q = G.dev_f16(b.q)
    lengths = seqs.lengths.clone()
    lengths[1] = 0
    y = awq.attend(q, cache, seqs._replace(lengths=lengths))
    assert bool((y[1] == 0).all())
    b.check(y, "beside an empty sequence", rows=[0, 2])
    # more rows than tokens: the first have no place
    b = Batch([6, 2], [0, 30], 8, 2, 128, 16, seed=2)
    cache, seqs = b.device()
    lengths = seqs.lengths.clone()
    lengths[0] = 4
    b.lengths[0] = 4
    b.place[:6] = np.arange(6) - 2
    y = awq.attend(G.dev_f16(b.q), cache, seqs._replace(lengths=lengths))
    assert bool((y[:2] == 0).all())
    b.check(y, "rows without a place")


@pytest.mark.parametrize("new", [5, 40, 150])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_later_tokens_that_are_not_finite_stay_unseen(new, bad):
    """Keys and values of a sequence's last tokens are not numbers: the rows before see nothing of them."""
    for Hq, Hkv in ((8, 2), (4, 4)):
        b = Batch([new, 1], [21, 5], Hq, Hkv, 128, 16, seed=new)
        last = b.lengths[0] - 2
        for p in (last, last + 1):
            page, slot = b.tables[0, p // 16], p % 16
            b.k[page, :, slot, 3] = bad
            b.v[page, :, slot, ::5] = bad
        y = attend(b)
        b.check(y, f"{new} rows before {bad}", rows=[0, 1, new // 2, new - 3, new])


def test_a_value_that_is_not_finite_reaches_the_rows_that_see_it():
    b = Batch([40], [21], 8, 2, 128, 16)
    p = b.lengths[0] - 20
    page, slot = b.tables[0, p // 16], p % 16
    b.v[page, 1, slot, 5] = np.inf
    y = attend(b).cpu().numpy().astype(np.float64)
    b.v[page, 1, slot, 5] = 0
    seen = y[40 - 20:].reshape(20, 8, 128)
    assert np.all(np.isinf(seen[:, 4:, 5])) and np.all(np.isfinite(seen[:, :4]))
    assert np.all(np.isfinite(y[:40 - 20]))
    assert np.all(np.isfinite(np.delete(seen[:, 4:], 5, 2)))


def test_large_scores_and_scale():
    b = Batch([1, 3], [500, 200], 8, 2, 128, 16, scale=6.0)
    b.check(attend(b), "scores of a few hundred")
    b = Batch([1, 3], [500, 200], 8, 2, 128, 16)
    b.check(attend(b, scale=0.7), "another scale", scale=0.7)


def test_equal_scores_average_the_values():
    b = Batch([1, 70], [300, 0], 8, 2, 128, 16)
    b.q[:] = 0
    b.check(attend(b), "queries of 0")


def test_rising_scores():
    """Each key's score is above the one before: the running maximum moves at every step."""
    b = Batch([1, 1], [700, 90], 2, 1, 64, 16)
    for s in range(2):
        for j in range(b.lengths[s]):
            b.k[b.tables[s, j // 16], :, j % 16] = 0
            b.k[b.tables[s, j // 16], :, j % 16, 0] = j * 0.5
    b.q[:] = 0
    b.q.reshape(b.T, 2, 64)[:, :, 0] = 1.0
    b.check(attend(b, scale=1.0), "rising scores", scale=1.0)
    b.q.reshape(b.T, 2, 64)[:, :, 0] = -1.0
    b.check(attend(b, scale=1.0), "falling scores", scale=1.0)


def test_strides_streams_graphs_and_repetition():
    awq = G.lib()
    for b in (Batch([1] * 9, [60 * i for i in range(9)], 16, 2, 128, 16, shared=64),
              Batch([100, 30], [5, 300], 16, 2, 128, 16), Batch([2, 1, 3], [4000, 3, 70], 16, 2, 128, 16)):
        cache, seqs = b.device()
        q = G.dev_f16(b.q)
        wide = torch.full((b.T, 3 * 2048 + 8), 5.0, dtype=torch.float16, device="cuda")
        wide[:, 2048:4096] = q
        y0 = awq.attend(q, cache, seqs, shared=b.shared)
        out = wide[:, 4096:6144]
        awq.attend(wide[:, 2048:4096], cache, seqs, shared=b.shared, y=out)
        assert torch.equal(out, y0) and bool((wide[:, 6144:] == 5.0).all()) and bool((wide[:, :2048] == 5.0).all())
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            there = awq.attend(q, cache, seqs, shared=b.shared)
        side.synchronize()
        assert torch.equal(there, y0)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            captured = awq.attend(q, cache, seqs, shared=b.shared)
        lengths = seqs.lengths.clone()
        for i in range(4):
            captured.zero_()
            seqs.lengths.copy_(lengths - (i % 2) * (i + 1) // 2 * (lengths > 4 + max(b.new) + b.shared))
            graph.replay()
            eager = awq.attend(q, cache, seqs, shared=b.shared)
            torch.cuda.synchronize()
            assert torch.equal(captured, eager)


@pytest.mark.parametrize("Hq,Hkv,D,S", [(8, 2, 128, 16), (64, 8, 128, 32), (4, 4, 64, 16), (16, 1, 256, 64), (10, 2, 96, 16),
                                        (40, 1, 128, 16)])
def test_chosen_pages(Hq, Hkv, D, S):
    awq = G.lib()
    b = Batch([1, 3, 1, 2], [40 * S, 9 * S + 3, 5, S - 2], Hq, Hkv, D, S, pad=1, seed=D)
    cache, seqs = b.device()
    for count in (1, 4, 7, 50):
        chosen = np.full((b.T, Hkv, count), -1)
        for t in range(b.T - 1):
            have = int(b.place[t]) // S + 1
            for h in range(Hkv):
                n = min(have, int(b.rng.integers(1, count + 1)))
                chosen[t, h, :n] = b.rng.permutation(have)[:n]
        dev = torch.from_numpy(chosen.astype(np.int32)).cuda()
        y = torch.full((b.T, Hq * D), 7.0, dtype=torch.float16, device="cuda")
        awq.attend_pages(G.dev_f16(b.q), cache, seqs, dev, y=y)
        assert bool((y[-1] == 7.0).all())
        b.check(y, f"{count} pages of {S}, {Hq}/{Hkv} heads of {D}", chosen=chosen)


def test_chosen_pages_none_all_and_out_of_range():
    awq = G.lib()
    b = Batch([1, 2], [200, 90], 8, 2, 128, 16)
    cache, seqs = b.device()
    q = G.dev_f16(b.q)
    none = torch.full((3, 2, 5), -1, dtype=torch.int32, device="cuda")
    assert bool((awq.attend_pages(q, cache, seqs, none) == 0).all())
    full = torch.arange(16, dtype=torch.int32, device="cuda").expand(3, 2, 16).contiguous()
    y = awq.attend_pages(q, cache, seqs, full)  # pages past the place are not seen
    b.check(y, "all pages")
    full[:, :, 14] = 1 << 30
    full[:, :, 15] = -5
    b.check(awq.attend_pages(q, cache, seqs, full), "numbers of no page")


def test_no_tokens():
    awq = G.lib()
    b = Batch([1], [20], 8, 2, 128, 16)
    cache, seqs = b.device()
    q = G.dev_f16(b.q)[:0]
    assert awq.attend(q, cache, seqs).shape == (0, 1024)
    pages = torch.zeros((0, 2, 3), dtype=torch.int32, device="cuda")
    assert awq.attend_pages(q, cache, seqs, pages).shape == (0, 1024)
