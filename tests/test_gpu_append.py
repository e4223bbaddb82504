"""awq_append_kv: rotation against fp64, the cache's slots and nothing else, the pages' bounds bit for bit."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import cache_oracle as C
from tests import _gpu as G
from tests._cache import Batch

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def freqs(R, base=10000.0):
    return (base ** (-np.arange(0, R, 2) / max(R, 1))).astype(np.float32)


def bounds_of(k, used):
    """Bounds of each page's used slots (pages without any: zeros)."""
    out = np.zeros(k.shape[:2] + (2, k.shape[3]), np.float16)
    for p in np.flatnonzero(used.any(1)):
        out[p, :, 0], out[p, :, 1] = k[p][:, used[p]].min(1), k[p][:, used[p]].max(1)
    return out


def run(b, R, interleaved=False, positions=None, axes=None, bounds=True, in_place=False, ld=0, freq=None):
    """Appends b's new tokens to what stands before them, and checks every output."""
    awq = G.lib()
    Hq, Hkv, D, S, T, real = b.Hq, b.Hkv, b.D, b.S, b.T, sum(b.new)
    width = (Hq + 2 * Hkv) * D
    x = b.rng.standard_normal((T, width)).astype(np.float16)
    x[real:] = np.nan
    fresh = np.zeros(b.used.shape, bool)
    where = []
    for t in range(T):
        if b.seq[t] >= 0 and b.place[t] >= 0:
            page, slot = int(b.tables[b.seq[t], b.place[t] // S]), int(b.place[t] % S)
            if 0 <= page < b.k.shape[0]:
                fresh[page, slot] = True
                where.append((t, page, slot))
    before = b.used & ~fresh
    cache, seqs = b.device()
    low = bounds_of(b.k, before)
    if bounds:
        cache = cache._replace(bounds=G.dev_f16(low))
    freq = freqs(R) if freq is None else freq
    dev = torch.from_numpy(x).cuda()
    if ld:
        wide = torch.full((T, width + ld), 3.0, dtype=torch.float16, device="cuda")
        wide[:, :width] = dev
        dev = wide[:, :width]
    kw = dict(interleaved=interleaved)
    if positions is not None:
        kw["positions"] = torch.from_numpy(positions.astype(np.int32)).cuda()
    if axes is not None:
        kw["axes"] = torch.from_numpy(axes.astype(np.int32)).cuda()
    q = dev[:, :Hq * D] if in_place else torch.full((T, Hq * D), 7.0, dtype=torch.float16, device="cuda")
    got = awq.append_kv(dev, cache, seqs, torch.from_numpy(freq).cuda() if R else None, q=q, **kw)
    assert got is q
    at = b.place if positions is None else positions
    rows = x.reshape(T, Hq + 2 * Hkv, D)
    ref, e = C.rotate(rows[:real, :Hq + Hkv], at[:real], freq if R else [], interleaved, axes)
    e = e + np.abs(ref) * 2.0 ** -11 + 2.0 ** -25
    out = q.cpu().numpy().reshape(T, Hq, D).astype(np.float64)
    placed = np.flatnonzero(b.place[:real] >= 0)
    assert np.all(np.abs(out[placed] - ref[placed, :Hq]) <= e[placed, :Hq]), "queries"
    if not in_place:
        left = np.setdiff1d(np.arange(T), placed)
        assert np.all(out[left] == 7.0), "rows without a place were written"
    k, v = cache.k.cpu().numpy(), cache.v.cpu().numpy()
    for t, page, slot in where:
        assert np.all(np.abs(k[page, :, slot] - ref[t, Hq:]) <= e[t, Hq:]), f"key of row {t}"
        assert np.array_equal(v[page, :, slot].view(np.uint16), rows[t, Hq + Hkv:].view(np.uint16)), f"value of row {t}"
    for new, old in ((k, b.k), (v, b.v)):
        kept = ~fresh
        assert np.array_equal(new.transpose(0, 2, 1, 3)[kept].view(np.uint16),
                              old.transpose(0, 2, 1, 3)[kept].view(np.uint16)), "another slot was written"
    if bounds:
        # (compared as numbers: -0 and 0 are equal)
        assert np.array_equal(cache.bounds.cpu().numpy(), bounds_of(k, before | fresh)), "bounds"
    return q, cache


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (36, 36), (8, 1), (14, 2), (64, 8), (7, 7)])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_heads(Hq, Hkv, D):
    run(Batch([1, 2, 5], [0, 15, 33], Hq, Hkv, D, 16, pad=2, seed=Hq), D)


@pytest.mark.parametrize("S", [16, 32, 64, 128, 256])
def test_runs_of_pages(S):
    run(Batch([1, S - 1, S, S + 1, 2 * S + 7], [S - 1, 1, 0, S // 2, 3], 4, 2, 128, S, pad=1, seed=S), 128)


@pytest.mark.parametrize("B", [1, 2, 63, 64, 65, 200])
def test_batches(B):
    run(Batch([1 + i % 3 for i in range(B)], [(13 * i) % 40 for i in range(B)], 4, 2, 64, 16, pad=B % 2), 64)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(64, 32), (96, 16), (128, 0), (128, 64), (128, 112), (256, 128)])
def test_part_of_the_channels(D, R, interleaved):
    run(Batch([3, 20], [9, 0], 6, 2, D, 16), R, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
def test_axes(interleaved):
    b = Batch([30, 9], [4, 17], 8, 2, 128, 32, pad=1)
    positions = b.rng.integers(0, 4000, (b.T, 3))
    run(b, 128, interleaved, positions, np.arange(64) % 3)
    run(Batch([30, 9], [4, 17], 8, 2, 128, 32), 64, interleaved, positions[:39], np.repeat([0, 1, 2], [8, 12, 12]))
    run(Batch([3], [4], 8, 2, 128, 32), 128, interleaved, positions[:3, 0])
    run(Batch([3], [4], 8, 2, 128, 32), 128, interleaved, positions[:3, :1])


def test_far_positions():
    b = Batch([8], [0], 4, 2, 128, 16)
    positions = np.array([0, 1, -1, 1000, 131071, 1 << 20, (1 << 24) + 1, (1 << 31) - 1])
    run(b, 128, positions=positions)
    run(b, 128, positions=positions, freq=np.full(64, np.float32(1.5707964)))


def test_queries_in_place_and_strides():
    run(Batch([3, 1, 20], [9, 0, 15], 8, 2, 128, 16), 128, in_place=True, ld=8)
    run(Batch([3, 1, 20], [9, 0, 15], 8, 2, 128, 16), 128, ld=24)


def test_without_bounds():
    run(Batch([3, 1, 20], [9, 0, 15], 8, 2, 128, 16), 128, bounds=False)


def test_pages_out_of_range_are_not_written():
    b = Batch([20, 3], [9, 0], 8, 2, 128, 16)
    b.tables[0, 1] = 1 << 29
    b.tables[1, 0] = -1
    b.used[:] = False
    b.used[b.tables[0, 0], :9] = True
    run(b, 128)


def test_more_rows_than_tokens_and_empty_sequences():
    b = Batch([6, 2, 4], [0, 30, 0], 8, 2, 128, 16)
    b.lengths[0], b.lengths[2] = 4, 0
    b.place[:6] = np.arange(6) - 2
    b.place[8:] = np.arange(4) - 4
    b.used[b.tables[2, 0]] = False
    b.used[b.tables[0, 0], 4:] = False
    run(b, 128)


def test_one_token_at_a_time_is_a_prompt_at_once():
    awq = G.lib()
    b = Batch([37], [0], 4, 2, 128, 16)
    _, seqs = b.device()
    x = torch.from_numpy(b.rng.standard_normal((37, 8 * 128)).astype(np.float16)).cuda()
    freq = torch.from_numpy(freqs(128)).cuda()
    caches = []
    for steps in ([37], [1] * 37, [5, 16, 1, 15]):
        cache, _ = b.device()
        cache = cache._replace(bounds=torch.zeros((cache.k.shape[0], 2, 2, 128), dtype=torch.float16, device="cuda"))
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


def test_not_finite_keys_and_bounds():
    """NaN in a key leaves the bounds to the others; infinities are bounds."""
    awq = G.lib()
    b = Batch([3], [0], 2, 1, 64, 16)
    cache, seqs = b.device()
    cache = cache._replace(bounds=torch.zeros((cache.k.shape[0], 1, 2, 64), dtype=torch.float16, device="cuda"))
    x = b.rng.standard_normal((3, 4, 64)).astype(np.float16)
    x[1, 2, 5], x[2, 2, 6], x[0, 2, 7] = np.nan, np.inf, -np.inf
    awq.append_kv(torch.from_numpy(x.reshape(3, 256)).cuda(), cache, seqs)
    got = cache.bounds[int(b.tables[0, 0]), 0].cpu().numpy()
    k = x[:, 2].astype(np.float32)
    assert np.array_equal(got[0], np.nanmin(k, 0)) and np.array_equal(got[1], np.nanmax(k, 0))


def test_streams_and_graphs():
    awq = G.lib()
    b = Batch([1] * 5, [3, 15, 16, 40, 90], 8, 2, 128, 16)
    cache, seqs = b.device()
    cache = cache._replace(bounds=G.dev_f16(bounds_of(b.k, b.used)))
    freq = torch.from_numpy(freqs(128)).cuda()
    x = torch.from_numpy(b.rng.standard_normal((5, 12 * 128)).astype(np.float16)).cuda()
    eager = awq.append_kv(x, cache, seqs, freq)
    first = [t.clone() for t in cache]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        q = awq.append_kv(x, cache, seqs, freq)
    for _ in range(3):
        for t, kept in zip(cache, first):
            t.copy_(kept)
        q.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q, eager)
        for t, kept in zip(cache, first):
            assert torch.equal(t.view(torch.int16), kept.view(torch.int16))


def test_no_tokens():
    awq = G.lib()
    b = Batch([1], [20], 8, 2, 128, 16)
    cache, seqs = b.device()
    assert awq.append_kv(torch.zeros((0, 12 * 128), dtype=torch.float16, device="cuda"), cache, seqs).shape == (0, 1024)
