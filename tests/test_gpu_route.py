"""awq_route_experts against the definition: whole numbers equal, weights to fp32 accuracy; ties, masks, infinities,
strides, every lane-group size, one block and many."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import fused_oracle as F
from tests import _gpu as G

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def check(logits, top_k, renormalize, ld=None):
    awq = G.lib()
    T, E = logits.shape
    dev = torch.from_numpy(np.ascontiguousarray(logits)).cuda()
    if ld:
        wide = torch.full((T, ld), 1e4, dtype=dev.dtype, device="cuda")
        wide[:, :E] = dev
        dev = wide[:, :E]
    got = awq.route_experts(dev, top_k, renormalize)
    ids, weights, offsets, rows, positions = F.route(logits, top_k, renormalize)
    what = f"T={T} E={E} k={top_k} renormalize={renormalize} {logits.dtype}"
    for name, ref in (("ids", ids), ("offsets", offsets), ("rows", rows), ("positions", positions)):
        assert np.array_equal(getattr(got, name).cpu().numpy(), ref), f"{what}: {name}"
    # fp32: an exponential to 2 units in the last place, a sum of at most 1024 terms of one sign in a tree or in
    # order over top_k <= 64, and a division: (2 + 64 + 10 + 1) * 2^-24 bounds it
    w = got.weights.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(w - weights) <= 80 * 2.0 ** -24 * weights + 1e-37), what
    return got


def logits_of(T, E, seed, dtype=np.float32):
    rng = np.random.default_rng([5, T, E, seed])
    return (rng.standard_normal((T, E)) + 0.7 * rng.standard_normal((1, E))).astype(dtype)


@pytest.mark.parametrize("E", [1, 2, 5, 8, 9, 16, 31, 33, 60, 64, 65, 128, 200, 256, 300, 512, 1000, 1024])
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_expert_counts(E, dtype):
    for T in (1, 3, 70):
        check(logits_of(T, E, 1, dtype), min(E, 1 + (E + T) % 9), (T + E) % 2 == 0)


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 255, 256, 257, 511, 512, 513, 1000, 2500])
def test_token_counts(T):
    check(logits_of(T, 16, 2), 3, True)
    check(logits_of(T, 60, 3, np.float16), 4, False)


@pytest.mark.parametrize("T,E,k,dtype", [(33000, 6, 1, np.float16), (40001, 10, 2, np.float32)])
def test_more_blocks_than_one_block_adds_up(T, E, k, dtype):
    check(logits_of(T, E, 5, dtype), k, True)


@pytest.mark.parametrize("E,k", [(8, 8), (64, 64), (100, 64), (1024, 64)])
def test_many_choices(E, k):
    check(logits_of(40, E, 4), k, True)
    check(logits_of(300, E, 4), k, False)


@pytest.mark.parametrize("T", [5, 300])
def test_ties_go_to_the_lower_index(T):
    rng = np.random.default_rng(T)
    for E in (8, 40, 128, 1024):
        check(rng.integers(0, 3, (T, E)).astype(np.float16), min(E, 6), True)
        check(np.zeros((T, E), np.float32), 2, False)


@pytest.mark.parametrize("T", [40, 600])
@pytest.mark.parametrize("renormalize", [True, False])
def test_masks_and_infinities(T, renormalize):
    """Masked logits (-inf, NaN), tokens with fewer than top_k open experts and with none, +inf, and the type's
    lowest value, which is an ordinary logit."""
    rng = np.random.default_rng(T)
    for E, k in ((8, 2), (64, 6), (200, 5)):
        v = logits_of(T, E, 6)
        v[rng.random((T, E)) < 0.3] = -np.inf
        v[rng.random((T, E)) < 0.1] = np.nan
        v[::5] = -np.inf                       # tokens to skip
        v[1::7, :] = -np.inf
        v[1::7, E - 1] = 3.0                   # one open expert
        v[2::11, 3] = np.inf
        v[2::11, 5] = np.inf
        v[3::13] = np.finfo(np.float32).min
        v[4::17] = -np.inf
        v[4::17, 2] = np.finfo(np.float32).min
        got = check(v, k, renormalize)
        assert bool((got.ids[0] == -1).all()) and bool((got.weights[0] == 0).all())


def test_all_tokens_masked():
    for T in (3, 700):
        got = check(np.full((T, 12), -np.inf, np.float16), 2, True)
        assert int(got.offsets[-1]) == 0 and bool((got.rows == -1).all())


def test_all_tokens_on_one_expert():
    v = np.zeros((900, 32), np.float32)
    v[:, 17] = 5.0
    check(v, 1, True)


def test_strides_streams_and_repetition():
    check(logits_of(77, 24, 8), 3, True, ld=57)
    check(logits_of(400, 24, 9, np.float16), 3, True, ld=31)
    awq = G.lib()
    x = torch.from_numpy(logits_of(3000, 64, 10)).cuda()
    first = awq.route_experts(x, 6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = awq.route_experts(x, 6)
    side.synchronize()
    for a, b, c in zip(first, there, awq.route_experts(x, 6)):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("T", [1, 500])
def test_in_a_graph(T):
    awq = G.lib()
    x = torch.from_numpy(logits_of(T, 64, 11)).cuda()
    eager = awq.route_experts(x, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = awq.route_experts(x, 4)
    for _ in range(4):
        for t in out:
            t.zero_()
        graph.replay()
        awq.route_experts(x, 2)
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert torch.equal(a, b)
