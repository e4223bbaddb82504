"""awq_linear_experts and awq_combine_experts against the fp64 oracle: ragged and empty experts, one token and many,
masked tokens, odd shapes, both zero point modes, strides, graphs; and the whole block."""
from __future__ import annotations

import numpy as np
import pytest

import workloads
from oracle import awq_oracle as O
from oracle import fused_oracle as F
from tests import _fused as H
from tests import _gpu as G

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def logits_of(T, E, seed, skew=0.7):
    rng = np.random.default_rng([6, T, E, seed])
    return (rng.standard_normal((T, E)) + skew * rng.standard_normal((1, E))).astype(np.float32)


def device_route(awq, ref):
    return awq.ExpertRoute(*(torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in
                             (ref[0], ref[1].astype(np.float32), *ref[2:])))


def run_case(logits, k, N, K, g, zp, act, gated, bias, residual, seed=0):
    """Both products of one routing: rows out, and rows combined."""
    awq = G.lib()
    T, E = logits.shape
    ref = F.route(logits, k, True)
    ids, weights, offsets, rows, positions = ref
    route = device_route(awq, ref)
    pe, wdq = H.packed_experts(awq, E, N, K, g, zp, seed)
    what = f"T={T} E={E} k={k} N={N} K={K} g={g} zp={zp} {act} gated={gated} bias={bias} residual={residual}"
    X = workloads.activations(T, K, cfg=12, layer=seed % 1000)
    b = H.halves((E, N), seed + 1) if bias else None
    bd = None if b is None else G.dev_f16(b)
    used = int(offsets[-1])
    y = torch.full((T * k, N // 2 if gated else N), 55.0, dtype=torch.float16, device="cuda")
    awq.linear_experts(G.dev_f16(X), pe, route, bd, act, gated, y=y)
    got = G.host_f16(y)
    H.check(got[:used], *F.linear_experts(X, wdq, offsets, rows, k, b, act, gated), "rows " + what)
    assert np.all(got[used:] == 55.0), what
    h = workloads.activations(T * k, K, cfg=12, layer=(seed + 5) % 1000)
    r = H.halves((T, N), seed + 2) if residual else None
    c = awq.combine_experts(G.dev_f16(h), pe, route, bd, None if r is None else G.dev_f16(r))
    H.check(G.host_f16(c), *F.combine_experts(h, wdq, offsets, positions, weights.astype(np.float32), b, r),
            "combined " + what)


@pytest.mark.parametrize("T", [1, 2, 3, 5, 9, 16, 33, 70, 150])
@pytest.mark.parametrize("gated", [False, True])
def test_token_counts(T, gated):
    run_case(logits_of(T, 8, T), 2, 144, 256, 64, True, "silu", gated, T % 2 == 1, T % 3 == 1, seed=T)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (40, 1, 1), (1, 16, 4), (7, 64, 6), (30, 100, 8), (90, 130, 3),
                                   (400, 4, 2), (700, 3, 1), (1, 64, 64)])
def test_expert_counts(T, E, k):
    run_case(logits_of(T, E, 3), k, 72, 96, 32, E % 2 == 0, "relu", False, True, True, seed=E)


@pytest.mark.parametrize("N,K,g", [(8, 32, 32), (16, 544, 32), (48, 64, 64), (264, 1088, 64), (520, 256, 256),
                                   (96, 2080, 32)])
@pytest.mark.parametrize("T", [1, 6, 50, 200])
def test_ragged_shapes(T, N, K, g):
    run_case(logits_of(T, 8, 4), 2, N, K, g, T != 6, "gelu_tanh", N % 16 == 0, False, T == 6, seed=N)


@pytest.mark.parametrize("T", [1, 4, 40, 300])
def test_every_token_on_one_expert_and_empty_ones(T):
    v = np.full((T, 12), -1.0, np.float32)
    v[:, 7] = 4.0
    run_case(v, 1, 128, 256, 128, True, "silu", True, False, True, seed=1)


@pytest.mark.parametrize("T", [1, 3, 20, 130])
def test_masked_tokens_and_short_choices(T):
    """Tokens routed nowhere (their output is the residual, or 0) and with fewer than top_k experts."""
    v = logits_of(T, 6, 8)
    v[::4] = -np.inf
    v[1::5, 1:] = -np.inf
    for residual in (False, True):
        run_case(v, 3, 80, 128, 64, True, "silu", False, True, residual, seed=2)


def test_all_tokens_masked():
    run_case(np.full((5, 6), -np.inf, np.float32), 2, 48, 64, 32, True, "none", True, False, True, seed=3)


def test_more_tokens_than_a_grid_has_rows():
    run_case(logits_of(33000, 4, 5), 2, 16, 32, 32, True, "silu", True, True, True, seed=4)


@pytest.mark.parametrize("T,E,k,N,K,gated", [(1, 8, 2, 22016, 4096, True), (1, 8, 2, 4096, 11008, False),
                                             (48, 64, 6, 2816, 2048, True), (300, 8, 2, 4096, 11008, False),
                                             (900, 8, 2, 4096, 4096, True)])
def test_large_layers(T, E, k, N, K, gated):
    """Full-size experts, a sample of output octets against the oracle."""
    awq = G.lib()
    g = 128
    gen = torch.Generator(device="cuda").manual_seed(T)
    w = (torch.randn((E, N, K), generator=gen, device="cuda") / K ** 0.5).half()
    pe = awq.pack_experts(w, g, True)
    del w
    logits = logits_of(T, E, 9)
    ids, weights, offsets, rows, positions = F.route(logits, k, True)
    route = awq.route_experts(torch.from_numpy(logits).cuda(), k)
    width = N // 2 if gated else N
    octets = np.sort(np.random.default_rng(T).choice(width // 8, 4, replace=False))
    cols = (octets[:, None] * 8 + np.arange(8)).reshape(-1)
    wr = np.concatenate([cols, width + cols]) if gated else cols
    qw, sc, qz = G.host_u32(pe.qweight), G.host_f16_bits(pe.scales), G.host_u32(pe.qzeros)

    def decoded(e):
        o = wr[::8] // 8
        return O.dequant_packed(qw[e][wr], sc[e][o], qz[e][o], len(wr), K, g, True)

    wdq = [decoded(e) for e in range(E)]
    if gated:
        X = workloads.activations(T, K, cfg=12, layer=7)
        y = G.host_f16(awq.linear_experts(G.dev_f16(X), pe, route, activation="silu", gated=True))
        H.check(y[:, cols], *F.linear_experts(X, wdq, offsets, rows, k, None, "silu", True), f"T={T} {K}->{N}")
    else:
        h = workloads.activations(T * k, K, cfg=12, layer=7)
        r = H.halves((T, N), 1)
        y = G.host_f16(awq.combine_experts(G.dev_f16(h), pe, route, residual=G.dev_f16(r)))
        H.check(y[:, cols], *F.combine_experts(h, wdq, offsets, positions, weights.astype(np.float32), None,
                                               r[:, cols]), f"T={T} {K}->{N}")


@pytest.mark.parametrize("T", [1, 5, 60])
def test_strides(T):
    awq = G.lib()
    E, k, N, K = 6, 2, 96, 160
    ref = F.route(logits_of(T, E, 2), k, True)
    route = device_route(awq, ref)
    pe, wdq = H.packed_experts(awq, E, N, K, 32, True, 4)
    X, h, r = (workloads.activations(n, K, cfg=12, layer=4) for n in (T, T * k, T))
    r = r[:, :N]

    def wide(a, pad):
        t = torch.full((a.shape[0], a.shape[1] + pad), float("nan"), dtype=torch.float16, device="cuda")
        t[:, 8:8 + a.shape[1]] = G.dev_f16(a)
        return t[:, 8:8 + a.shape[1]]

    for gated in (False, True):
        width = N // 2 if gated else N
        big = torch.full((T * k, width + 16), 3.0, dtype=torch.float16, device="cuda")
        awq.linear_experts(wide(X, 24), pe, route, None, "silu", gated, y=big[:, 8:8 + width])
        H.check(G.host_f16(big[:, 8:8 + width].contiguous()),
                *F.linear_experts(X, wdq, ref[2], ref[3], k, None, "silu", gated), f"strided T={T}")
        assert bool((big[:, :8] == 3.0).all()) and bool((big[:, 8 + width:] == 3.0).all())
    big = torch.full((T, N + 16), 3.0, dtype=torch.float16, device="cuda")
    awq.combine_experts(wide(h, 40), pe, route, None, wide(r, 16), y=big[:, 8:8 + N])
    H.check(G.host_f16(big[:, 8:8 + N].contiguous()),
            *F.combine_experts(h, wdq, ref[2], ref[4], ref[1].astype(np.float32), None, r), f"strided combine T={T}")
    assert bool((big[:, :8] == 3.0).all()) and bool((big[:, 8 + N:] == 3.0).all())
    # the residual stream updated in place
    stream = G.dev_f16(r)
    apart = awq.combine_experts(G.dev_f16(h), pe, route, residual=stream)
    awq.combine_experts(G.dev_f16(h), pe, route, residual=stream, y=stream)
    assert torch.equal(apart, stream)


def test_pack_experts_is_pack_expert_by_expert():
    awq = G.lib()
    W = torch.stack([G.dev_f16(workloads.weight(40, 256, cfg=12, layer=e)) for e in range(5)])
    for zp in (True, False):
        pe = awq.pack_experts(W, 64, zp)
        assert (pe.E, pe.N, pe.K) == (5, 40, 256)
        for e in range(5):
            one = awq.pack(W[e].contiguous(), 64, zp)
            assert torch.equal(pe.qweight[e], one.qweight) and torch.equal(pe.scales[e], one.scales)
            assert (pe.qzeros is None) if not zp else torch.equal(pe.qzeros[e], one.qzeros)
        listed = awq.pack_experts([W[e] for e in range(5)], 64, zp)
        assert torch.equal(listed.qweight, pe.qweight)


@pytest.mark.parametrize("T", [1, 6, 40, 500])
def test_expert_mlp_is_its_three_steps_and_repeats(T):
    """The whole block: the steps' composition, the same bits again, on another stream and in a graph."""
    awq = G.lib()
    E, k, K, Fw = 8, 2, 256, 320
    up, wup = H.packed_experts(awq, E, 2 * Fw, K, 64, True, 31)
    down, wdn = H.packed_experts(awq, E, K, Fw, 32, True, 41)
    X, r, v = workloads.activations(T, K, cfg=12, layer=T % 1000), H.halves((T, K), T), logits_of(T, E, 12)
    x, res, lg = G.dev_f16(X), G.dev_f16(r), torch.from_numpy(v).cuda()
    y = awq.expert_mlp(x, lg, up, down, k, residual=res)
    route = awq.route_experts(lg, k)
    h = awq.linear_experts(x, up, route, activation="silu", gated=True)
    assert torch.equal(y, awq.combine_experts(h, down, route, residual=res))
    ids, weights, offsets, rows, positions = F.route(v, k, True)
    H.check(G.host_f16(h), *F.linear_experts(X, wup, offsets, rows, k, None, "silu", True), f"block T={T}")
    H.check(G.host_f16(y), *F.combine_experts(G.host_f16(h), wdn, offsets, positions, weights.astype(np.float32),
                                              None, r), f"block T={T}")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = awq.expert_mlp(x, lg, up, down, k, residual=res)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = awq.expert_mlp(x, lg, up, down, k, residual=res)
    side.synchronize()
    assert torch.equal(y, there)
    for _ in range(4):
        out.zero_()
        graph.replay()
        assert torch.equal(awq.expert_mlp(x, lg, up, down, k, residual=res), y)
        torch.cuda.synchronize()
        assert torch.equal(out, y)
