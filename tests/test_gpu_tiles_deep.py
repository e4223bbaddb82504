"""The matrix-core tiles where a workgroup takes several tiles of several K steps (an odd and an even number of them, and
half a step at the end): the next tile's first loads under the epilogue of the one before, the tallest tiles first and
every other round backwards, more than 64 experts.  Every row, and one octet of columns of every column tile."""
from __future__ import annotations

import numpy as np
import pytest

import workloads
from oracle import awq_oracle as O
from oracle import fused_oracle as F
from tests import _fused as H
from tests import _gpu as G
from tests.test_gpu_experts import logits_of

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def experts(awq, E, N, K, g, zp):
    gen = torch.Generator(device="cuda").manual_seed(N + K)
    return awq.pack_experts((torch.randn((E, N, K), generator=gen, device="cuda") / K ** 0.5).half(), g, zp)


def sampled(width, step):
    """One octet of every `step` columns, at another place each."""
    firsts = np.arange(0, width, step)
    octets = (firsts + 8 * (np.arange(len(firsts)) * 5 % (step // 8))) // 8
    octets = octets[octets < width // 8]
    return (octets[:, None] * 8 + np.arange(8)).reshape(-1)


def decoded(pe, rows):
    qw, sc = G.host_u32(pe.qweight), G.host_f16_bits(pe.scales)
    qz = G.host_u32(pe.qzeros) if pe.zero_point else None
    o = rows[::8] // 8
    return [O.dequant_packed(qw[e][rows], sc[e][o], qz[e][o] if pe.zero_point else None, len(rows), pe.K, pe.group_size,
                             pe.zero_point) for e in range(pe.E)]


# (E, T): 8 experts of 375 rows on average, 70 of 69 and 130 of 71; 5, 6 and 4 1/2 steps
@pytest.mark.parametrize("E,T,N", [(8, 1500, 8192), (70, 2400, 2048), (130, 4600, 1024)])
@pytest.mark.parametrize("K,g,zp", [(320, 64, True), (384, 128, False), (288, 32, True)])
def test_rounds_of_expert_tiles(E, T, N, K, g, zp):
    awq = G.lib()
    k = 2
    logits = logits_of(T, E, 41)
    ids, weights, offsets, rows, positions = F.route(logits, k, True)
    route = awq.route_experts(torch.from_numpy(logits).cuda(), k)
    pe = experts(awq, E, N, K, g, zp)
    X = workloads.activations(T, K, cfg=12, layer=41)
    what = f"E={E} T={T} {K} -> {N} g={g}"
    for gated in (True, False):
        width = N // 2 if gated else N
        cols = sampled(width, 128)
        wr = np.concatenate([cols, width + cols]) if gated else cols
        y = G.host_f16(awq.linear_experts(G.dev_f16(X), pe, route, activation="silu", gated=gated))
        H.check(y[:, cols], *F.linear_experts(X, decoded(pe, wr), offsets, rows, k, None, "silu", gated),
                f"{what} gated={gated}")
    h, r = workloads.activations(T * k, K, cfg=12, layer=42), H.halves((T, N), 42)
    cols = sampled(N, 256)
    y = G.host_f16(awq.combine_experts(G.dev_f16(h), pe, route, residual=G.dev_f16(r)))
    H.check(y[:, cols], *F.combine_experts(h, decoded(pe, cols), offsets, positions, weights.astype(np.float32), None,
                                           r[:, cols]), f"{what} combined")


@pytest.mark.parametrize("K,g", [(320, 64), (384, 128), (288, 32)])
@pytest.mark.parametrize("gated", [False, True])
def test_rounds_of_one_layer_tiles(K, g, gated):
    awq = G.lib()
    M, N = 1100, 22016
    pe = experts(awq, 1, N, K, g, True)
    pw = awq.PackedWeight(pe.qweight[0], pe.scales[0], pe.qzeros[0], N, K, g, True)
    width = N // 2 if gated else N
    cols = sampled(width, 128 if gated else 256)
    wr = np.concatenate([cols, width + cols]) if gated else cols
    X, b, r = workloads.activations(M, K, cfg=11, layer=43), H.halves(N, 43), H.halves((M, width), 44)
    y = G.host_f16(awq.linear_fused(G.dev_f16(X), pw, G.dev_f16(b), "silu", gated, G.dev_f16(r)))
    H.check(y[:, cols], *F.linear_fused(X, decoded(pe, wr)[0], b[wr], "silu", gated, r[:, cols]),
            f"{M} x {K} -> {N} gated={gated}")


@pytest.mark.parametrize("K,g", [(384, 128), (320, 64), (288, 32)])
def test_same_bits_again_on_another_stream_and_in_a_graph(K, g):
    """Several rounds of tiles of ragged experts, and their weighted sum."""
    awq = G.lib()
    E, T, N, k = 8, 1500, 8192, 2
    pe = experts(awq, E, N, K, g, True)
    route = awq.route_experts(torch.from_numpy(logits_of(T, E, 45)).cuda(), k)
    x = G.dev_f16(workloads.activations(T, K, cfg=12, layer=45))
    h = G.dev_f16(workloads.activations(T * k, K, cfg=12, layer=46))

    def both():
        return (awq.linear_experts(x, pe, route, activation="silu", gated=True), awq.combine_experts(h, pe, route))

    first = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = both()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = both()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, there))
    for _ in range(4):
        for t in out:
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(first, both()))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, out))
