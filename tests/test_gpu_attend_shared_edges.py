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


def test_a_first_sequence_that_empties_between_replays():
    """Captured with rows in every sequence; replayed without any in the first, and its table of no page."""
    awq = G.lib()
    for D, new in ((128, 1), (256, 2), (128, 60)):
        b = Batch([new] * 3, [9, 30, 4], 8, 2, D, 16, shared=160, seed=new)
        cache, seqs = b.device()
        q = G.dev_f16(b.q)
        eager = awq.attend(q, cache, seqs, shared=160)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y = awq.attend(q, cache, seqs, shared=160)
        kept = [t.clone() for t in seqs]
        for empty in (False, True, False, True):
            for t, was in zip(seqs, kept):
                t.copy_(was)
            if empty:
                seqs.offsets[0] = new
                seqs.lengths[0] = 0
                seqs.tables[0] = -1
            y.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y[new:], eager[new:]), (D, new, empty)
            assert bool((y[:new] == 7.0).all()) if empty else torch.equal(y[:new], eager[:new]), (D, new, empty)
