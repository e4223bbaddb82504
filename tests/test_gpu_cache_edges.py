"""The paged cache's operators where a batch is unusual: more sequences than lanes, empty ones among them, rows before the
first sequence, numbers that contradict each other, offsets past 32 bits, a caller's own workspace, two host threads at
once, a block captured into a graph."""
from __future__ import annotations

import threading

import numpy as np
import pytest

from tests import _gpu as G
from tests._cache import Batch
from tests._fused import halves, packed_layer

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).cuda()


def output(b):
    return torch.full((b.T, b.Hq * b.D), 7.0, dtype=torch.float16, device="cuda")


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("shared", [0, 160])
@pytest.mark.parametrize("new", [[1] * 130, [0, 1, 0, 3, 2] * 29, [0] * 70 + [40, 0, 9] + [0] * 60 + [33]])
def test_many_sequences(new, shared, D):
    awq = G.lib()
    b = Batch(new, [(13 * i) % 90 for i in range(len(new))], 8, 2, D, 16, shared=shared, pad=2, seed=len(new))
    cache, seqs = b.device()
    y = output(b)
    awq.attend(G.dev_f16(b.q), cache, seqs, shared=shared, y=y)
    assert bool((y[sum(new):] == 7.0).all())
    b.check(y, f"{len(new)} sequences, {shared} shared, heads of {D}")


@pytest.mark.parametrize("new,shared", [([1, 1, 1], 0), ([1, 2, 1], 64), ([70, 3], 0), ([70, 3], 64)])
def test_rows_before_the_first_sequence(new, shared):
    awq = G.lib()
    b = Batch(new, [50, 0, 17][:len(new)], 8, 2, 128, 16, shared=shared, pad=1)
    cache, seqs = b.device()
    plain = output(b)
    awq.attend(G.dev_f16(b.q), cache, seqs, shared=shared, y=plain)
    q = np.concatenate([np.full((3, b.q.shape[1]), np.nan, np.float16), b.q])
    later = seqs._replace(offsets=i32(b.offsets + 3))
    y = torch.full((b.T + 3, b.Hq * b.D), 7.0, dtype=torch.float16, device="cuda")
    awq.attend(G.dev_f16(q), cache, later, shared=shared, y=y)
    assert bool((y[:3] == 7.0).all()) and bool((y[3 + sum(new):] == 7.0).all())
    b.check(y[3:], "behind rows of no sequence")
    if shared == 0:
        pages = torch.arange(40, dtype=torch.int32, device="cuda").expand(b.T + 3, 2, 40).contiguous()
        y.fill_(7.0)
        awq.attend_pages(G.dev_f16(q), cache, later, pages, y=y)
        assert bool((y[:3] == 7.0).all()) and bool((y[3 + sum(new):] == 7.0).all())
        b.check(y[3:], "chosen pages behind rows of no sequence")


def test_lengths_past_the_table_end_at_it():
    awq = G.lib()
    b = Batch([1, 2, 40], [47, 46, 24], 8, 2, 128, 16, width=4)  # (64 places each: lengths 48, 48, 64)
    b.lengths[0], b.lengths[1] = 48, 48
    cache, seqs = b.device()
    q = G.dev_f16(b.q)
    most = seqs._replace(tables=seqs.tables[:, :3].contiguous())
    for lengths in ([48, 48, 48], [49, 5000, 1 << 30], [(1 << 31) - 1, 48, 48]):
        y = awq.attend(q, cache, most._replace(lengths=i32(lengths)))
        z = awq.attend(q, cache, most._replace(lengths=i32([48, 48, 48])))
        assert torch.equal(y, z)


@pytest.mark.parametrize("offsets", [[0, 2, 1, 3], [0, 3, 3, 1], [2, 1, 0, 3], [-5, 1, 2, 900], [7, -7, 7, -7]])
def test_offsets_out_of_order_stay_within_the_buffers(offsets):
    """Wrong results, but of the right places: what stands around the output and the cache is as it was."""
    awq = G.lib()
    b = Batch([1, 1, 1], [30, 70, 5], 8, 2, 128, 16)
    cache, seqs = b.device()
    bad = seqs._replace(offsets=i32(offsets))
    wide = torch.full((5, 1024 + 16), 7.0, dtype=torch.float16, device="cuda")
    for shared in (0, 16):
        awq.attend(G.dev_f16(b.q), cache, bad, shared=shared, y=wide[1:4, 8:1032])
        assert bool((wide[0] == 7).all()) and bool((wide[4] == 7).all()) and bool((wide[:, :8] == 7).all())
        assert bool((wide[:, 1032:] == 7).all())
    bounds = torch.zeros((b.k.shape[0], 2, 2, 128), dtype=torch.float16, device="cuda")
    chosen = awq.select_pages(G.dev_f16(b.q), cache._replace(bounds=bounds), bad, 2)
    awq.attend_pages(G.dev_f16(b.q), cache, bad, chosen, y=wide[1:4, 8:1032])
    assert bool((wide[0] == 7).all()) and bool((wide[4] == 7).all())


def test_heads_at_their_limit():
    awq = G.lib()
    for Hq, Hkv in ((1024, 1), (1024, 1024), (999, 3)):
        b = Batch([1, 2], [40, 3], Hq, Hkv, 64, 16, seed=Hkv)
        cache, seqs = b.device()
        b.check(awq.attend(G.dev_f16(b.q), cache, seqs), f"{Hq}/{Hkv} heads", rows=[1])


def test_a_long_prompt():
    awq = G.lib()
    b = Batch([4099], [0], 4, 2, 64, 64)
    cache, seqs = b.device()
    b.check(awq.attend(G.dev_f16(b.q), cache, seqs), "a prompt of 4099", rows=[0, 31, 32, 127, 128, 2000, 4097, 4098])


def test_offsets_past_32_bits():
    """A cache of more than 2^31 elements whose last pages are used: appending, both ways of attending, selecting."""
    awq = G.lib()
    pages, Hkv, S, D = 33000, 8, 64, 128
    b = Batch([1, 3, 1], [700, 5, 130], 16, Hkv, D, S, seed=9)
    pool = b.k.shape[0]
    small, seqs = b.device()
    big = awq.KvCache(*(torch.empty((pages, Hkv, S, D), dtype=torch.float16, device="cuda") for _ in range(2)),
                      torch.zeros((pages, Hkv, 2, D), dtype=torch.float16, device="cuda"))
    assert (pages - pool) * Hkv * S * D > 1 << 31
    big.k[pages - pool:], big.v[pages - pool:] = small.k, small.v
    used = [b.tables[s, i] for s in range(b.B) for i in range(-(-b.lengths[s] // S))]
    bounds = torch.zeros((pool, Hkv, 2, D), dtype=torch.float16, device="cuda")
    for p in used:
        live = small.k[int(p)][:, torch.from_numpy(b.used[p]).cuda()]
        bounds[int(p), :, 0], bounds[int(p), :, 1] = live.amin(1), live.amax(1)
    big.bounds[pages - pool:] = bounds
    inside = (b.tables >= 0) & (b.tables < pool)
    far = seqs._replace(tables=i32(np.where(inside, b.tables + pages - pool, -1)))
    q = G.dev_f16(b.q)
    assert torch.equal(awq.attend(q, big, far), awq.attend(q, small, seqs))
    many = Batch([90], [300], 16, Hkv, D, S, seed=10)  # row tiles
    at = pages - many.k.shape[0]
    big.k[at:], big.v[at:] = G.dev_f16(many.k), G.dev_f16(many.v)
    cache, one = many.device()
    shifted = one._replace(tables=i32(np.where((many.tables >= 0) & (many.tables < many.k.shape[0]), many.tables + at, -1)))
    mq = G.dev_f16(many.q)
    assert torch.equal(awq.attend(mq, big, shifted), awq.attend(mq, cache, one))
    # (the first batch's pages again)
    big.k[pages - pool:], big.v[pages - pool:] = small.k, small.v
    small = small._replace(bounds=bounds.clone())
    chosen = awq.select_pages(q, big, far, 4)
    assert torch.equal(chosen, awq.select_pages(q, small, seqs, 4))
    assert torch.equal(awq.attend_pages(q, big, far, chosen), awq.attend_pages(q, small, seqs, chosen))
    x = torch.from_numpy(b.rng.standard_normal((b.T, 32 * D)).astype(np.float16)).cuda()
    freq = torch.from_numpy((100.0 ** (-np.arange(0, D, 2) / D)).astype(np.float32)).cuda()
    assert torch.equal(awq.append_kv(x, big, far, freq), awq.append_kv(x, small, seqs, freq))
    for got, want in zip(big, small):
        assert torch.equal(got[pages - pool:].view(torch.int16), want.view(torch.int16))


def test_workspace_of_the_caller():
    awq = G.lib()
    lib = awq.load_library()
    for new, shared in (([1, 1], 0), ([1] * 40, 640), ([40, 60], 0)):
        b = Batch(new, [(31 * i) % 600 for i in range(len(new))], 16, 2, 128, 16, shared=shared)
        cache, seqs = b.device()
        q = G.dev_f16(b.q)
        need = lib.awq_attend_workspace_bytes(b.T, b.B, 16, 2, 128, b.width, 16, shared)
        ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
        y = awq.attend(q, cache, seqs, shared=shared, workspace=ws[:need])
        assert torch.equal(y, awq.attend(q, cache, seqs, shared=shared)) and bool((ws[need:] == 255).all())
        if need:
            with pytest.raises(awq.AwqError):
                awq.attend(q, cache, seqs, shared=shared, workspace=ws[:need - 1])
            with pytest.raises(awq.AwqError):
                awq.attend(q, cache, seqs, shared=shared, workspace=ws[1:])


def test_two_host_threads_at_once():
    awq = G.lib()
    jobs = []
    for i, (new, shared) in enumerate((([1] * 20, 320), ([1, 1, 1], 0), ([50, 20], 0))):
        b = Batch(new, [(97 * j) % 900 for j in range(len(new))], 16, 2, 128, 16, shared=shared, seed=i)
        cache, seqs = b.device()
        q = G.dev_f16(b.q)
        jobs.append((q, cache, seqs, shared, awq.attend(q, cache, seqs, shared=shared)))
    torch.cuda.synchronize()
    wrong, failed = [], []

    def work(first):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                got = [(i, awq.attend(q, cache, seqs, shared=shared))
                       for n in range(12) for i, (q, cache, seqs, shared, _) in [((first + n) % 3, jobs[(first + n) % 3])]]
            stream.synchronize()
            wrong.extend(i for i, y in got if not torch.equal(y, jobs[i][4]))
        except Exception as e:  # (of the thread: raised below)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and not wrong, (failed, wrong)


@pytest.mark.parametrize("mode", ["all", "shared", "pages"])
def test_a_block_in_a_graph(mode):
    """A decoding step captured once and replayed as the sequences grow, against the same steps made one by one."""
    awq = G.lib()
    HQ, HKV, D, S, K, B = 8, 2, 64, 16, 256, 3
    pw, _ = packed_layer(awq, (HQ + 2 * HKV) * D, K, 128, True, 5)
    po, _ = packed_layer(awq, K, HQ * D, 64, False, 6)
    freq = torch.from_numpy((10000.0 ** (-np.arange(0, D, 2) / D)).astype(np.float32)).cuda()
    tables = np.random.default_rng(1).permutation(60).reshape(B, 20)
    tables[:, :4] = tables[0, :4]
    kw = {"shared": 64} if mode == "shared" else {"pages": 3} if mode == "pages" else {}
    caches = [awq.kv_cache(60, HKV, D, S, bounds=True) for _ in range(2)]
    lengths = i32([64])
    prompt = torch.from_numpy(halves((64, K), 1)).cuda()
    for cache in caches:
        for t in (cache.k, cache.v, cache.bounds):
            t.zero_()
        awq.attention(prompt, pw, po, cache, awq.Sequences(i32([0, 64]), lengths, i32(tables[:1])), freq)
    x = torch.zeros((B, K), dtype=torch.float16, device="cuda")
    lengths = i32([64 + 1] * B)
    seqs = awq.Sequences(i32(range(B + 1)), lengths, i32(tables))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):  # (the capture below wants everything loaded; position 64 is written again)
        awq.attention(x, pw, po, caches[0], seqs, freq, **kw)
    stream.synchronize()
    caches[0].bounds[tables[:, 4]] = 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        captured = awq.attention(x, pw, po, caches[0], seqs, freq, **kw)
    for step in range(6):
        x.copy_(torch.from_numpy(halves((B, K), 20 + step)))
        graph.replay()
        eager = awq.attention(x, pw, po, caches[1], seqs, freq, **kw)
        torch.cuda.synchronize()
        assert torch.equal(captured, eager), step
        for got, want in zip(*caches):
            assert torch.equal(got, want)
        lengths += 1


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("new,past,shared", [(3, 200, 0), (6, 200, 0), (20, 200, 0), (150, 400, 0), (3, 200, 64), (40, 30, 160)])
def test_values_that_are_not_finite_reach_their_rows_only(new, past, shared, D):
    """An infinity and a NaN among the new tokens' values: rows before them are as without, rows from them on have them in
    their channels and nothing else."""
    awq = G.lib()
    b = Batch([new, 1], [past, 9], 8, 2, D, 16, shared=shared, seed=new)
    p = shared + past + new // 2
    page, slot = b.tables[0, p // 16], p % 16
    b.v[page, 1, slot, 5], b.v[page, 0, slot, D - 3] = np.inf, np.nan
    cache, seqs = b.device()
    q = G.dev_f16(b.q)
    results = [awq.attend(q, cache, seqs, shared=shared)]
    if shared == 0:
        pages = torch.arange(b.width, dtype=torch.int32, device="cuda").expand(b.T, 2, b.width).contiguous()
        results.append(awq.attend_pages(q, cache, seqs, pages))
    b.v[page, 1, slot, 5] = b.v[page, 0, slot, D - 3] = 0
    rows = sorted({0, new // 2 - 1, new // 2, new - 1, new})
    ref, bound, _ = b.expected(rows=rows)
    for y in results:
        got = y.cpu().numpy().astype(np.float64)[rows].reshape(len(rows), 8, D)
        for i, t in enumerate(rows):
            sees = new // 2 <= t < new
            assert np.all(np.isposinf(got[i, 4:, 5])) if sees else np.all(np.isfinite(got[i, 4:, 5])), (t, "infinity")
            assert np.all(np.isnan(got[i, :4, D - 3])) if sees else np.all(np.isfinite(got[i, :4, D - 3])), (t, "NaN")
            keep = np.ones((8, D), bool)
            if sees:
                keep[4:, 5] = keep[:4, D - 3] = False
            off = np.abs(got[i][keep] - ref[i].reshape(8, D)[keep])
            assert np.all(off <= bound[i].reshape(8, D)[keep]), (t, float(off.max()))


@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_rising_scores_at_every_head_size(D):
    """The running maximum moves at every block, in waves and in row tiles: sums are rescaled each time."""
    awq = G.lib()
    for new, past in ((1, 700), (5, 300), (70, 300)):
        b = Batch([new, 1], [past, 40], 4, 1, D, 16, seed=new)
        for s in range(2):
            for j in range(b.lengths[s]):
                b.k[b.tables[s, j // 16], :, j % 16] = 0
                b.k[b.tables[s, j // 16], :, j % 16, 0] = j * 0.5
        for sign in (1.0, -1.0):
            b.q[:] = 0
            b.q.reshape(b.T, 4, D)[:, :, 0] = sign
            cache, seqs = b.device()
            b.check(awq.attend(G.dev_f16(b.q), cache, seqs, scale=1.0), f"{new} rows, heads of {D}, {sign}", scale=1.0)
