"""awq_linear_fused against the fp64 oracle: token counts of every regime, ragged N and K, group sizes, both zero point
modes, every activation, gate, bias and residual; strides, aliasing, streams, graphs and offsets past 32 bits."""
from __future__ import annotations

import numpy as np
import pytest

import workloads
from oracle import fused_oracle as F
from tests import _fused as H
from tests import _gpu as G

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def run_case(M, N, K, g, zp, act, gated, bias, residual, seed=0):
    awq = G.lib()
    pw, wdq = H.packed_layer(awq, N, K, g, zp, seed)
    X = workloads.activations(M, K, cfg=11, layer=seed % 1000)
    b = H.halves(N, seed + 1) if bias else None
    r = H.halves((M, N // 2 if gated else N), seed + 2) if residual else None
    y = awq.linear_fused(G.dev_f16(X), pw, None if b is None else G.dev_f16(b), act, gated,
                         None if r is None else G.dev_f16(r))
    H.check(G.host_f16(y), *F.linear_fused(X, wdq, b, act, gated, r),
            f"M={M} N={N} K={K} g={g} zp={zp} {act} gated={gated} bias={bias} residual={residual}")


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9, 15, 16, 17, 31, 33, 48, 49, 64, 65, 100, 128, 129, 257, 300])
@pytest.mark.parametrize("gated", [False, True])
def test_token_counts(M, gated):
    run_case(M, 272, 512, 128, True, "silu", gated, True, True, seed=M)


@pytest.mark.parametrize("M", [1, 5, 13, 40, 90])
@pytest.mark.parametrize("N,K,g", [(8, 32, 32), (16, 96, 32), (24, 64, 64), (40, 160, 32), (264, 544, 32),
                                   (1032, 128, 128), (520, 768, 256), (72, 2080, 32), (136, 1088, 64)])
def test_ragged_shapes(M, N, K, g):
    zp = bool((N + M) & 8)
    run_case(M, N, K, g, zp, "none", False, M == 13, M == 40, seed=N + K)
    if N % 16 == 0:
        run_case(M, N, K, g, not zp, "gelu", True, M != 13, False, seed=N + K + 1)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M", [1, 6, 30, 70])
def test_activations(M, gated, act):
    run_case(M, 128, 256, 64, M != 6, act, gated, True, gated, seed=len(act) + M)


@pytest.mark.parametrize("M,N,K,gated", [(1, 4096, 4096, False), (1, 22016, 4096, True), (1, 4096, 11008, False),
                                         (7, 4096, 11008, False), (3, 22016, 4096, True), (13, 4096, 11008, False),
                                         (61, 11008, 4096, False), (32, 8192, 4096, True), (200, 4096, 4096, False)])
def test_7b_layers(M, N, K, gated):
    """Full-size layers, a sample of output octets against the oracle."""
    awq = G.lib()
    g = 128
    gen = torch.Generator(device="cuda").manual_seed(N + M)
    w = (torch.randn((N, K), generator=gen, device="cuda") / K ** 0.5).half()
    pw = awq.pack(w, g, True)
    X = workloads.activations(M, K, cfg=11, layer=M)
    b = H.halves(N, 3)
    width = N // 2 if gated else N
    r = H.halves((M, width), 4)
    y = G.host_f16(awq.linear_fused(G.dev_f16(X), pw, G.dev_f16(b), "silu", gated, G.dev_f16(r)))
    octets = np.sort(np.random.default_rng(M).choice(width // 8, 12, replace=False))
    cols = (octets[:, None] * 8 + np.arange(8)).reshape(-1)
    wr = np.concatenate([cols, width + cols]) if gated else cols
    wdq = awq.awq_dequant(pw.qweight, pw.scales, pw.qzeros, N, K, g, True)
    del wdq  # (rounded to fp16: the oracle decodes the sampled rows itself)
    from oracle import awq_oracle as O

    qw, sc, qz = G.host_u32(pw.qweight), G.host_f16_bits(pw.scales), G.host_u32(pw.qzeros)
    full = {}
    for o in np.unique(wr // 8):
        full[o] = O.dequant_packed(qw[8 * o:8 * o + 8], sc[o:o + 1], qz[o:o + 1], 8, K, g, True)
    W = np.concatenate([full[n // 8][n % 8][None] for n in wr])
    ref, bound = F.linear_fused(X, W, b[wr], "silu", gated, r[:, cols])
    H.check(y[:, cols], ref, bound, f"M={M} {K}->{N} gated={gated}")


def test_prefill_tiles():
    """Several 256-row tiles with ragged edges in both directions, gated and not."""
    for gated, N in ((False, 1096), (True, 1104)):
        run_case(700, N, 1088, 64, True, "silu", gated, True, True, seed=5)


@pytest.mark.parametrize("M", [1, 4, 12, 40, 150])
@pytest.mark.parametrize("gated", [False, True])
def test_strides_and_guard_columns(M, gated):
    """Rows of x, residual and y at strides of their own; nothing beyond y's columns is written."""
    awq = G.lib()
    N, K, g = 144, 224, 32
    width = N // 2 if gated else N
    pw, wdq = H.packed_layer(awq, N, K, g, True, 7)
    X, r = workloads.activations(M, K, cfg=11, layer=8), H.halves((M, width), 9)
    big_x = torch.full((M, K + 72), float("nan"), dtype=torch.float16, device="cuda")
    big_x[:, 8:8 + K] = G.dev_f16(X)
    big_r = torch.full((M, width + 40), float("nan"), dtype=torch.float16, device="cuda")
    big_r[:, 16:16 + width] = G.dev_f16(r)
    big_y = torch.full((M + 1, width + 24), 77.0, dtype=torch.float16, device="cuda")
    y = big_y[:M, 8:8 + width]
    out = awq.linear_fused(big_x[:, 8:8 + K], pw, None, "relu", gated, big_r[:, 16:16 + width], y=y)
    assert out.data_ptr() == y.data_ptr()
    H.check(G.host_f16(y.contiguous()), *F.linear_fused(X, wdq, None, "relu", gated, r), f"strided M={M}")
    big_y[:M, 8:8 + width] = 77.0
    assert bool((big_y == 77.0).all()), "written outside y"


@pytest.mark.parametrize("M", [1, 8, 24, 64, 260])
def test_residual_in_place(M):
    """y may be the residual itself, and the result is that of a separate one, bit for bit."""
    awq = G.lib()
    pw, _ = H.packed_layer(awq, 264, 512, 128, True, 3)
    x, r = G.dev_f16(workloads.activations(M, 512, cfg=11, layer=3)), G.dev_f16(H.halves((M, 264), 3))
    apart = awq.linear_fused(x, pw, residual=r)
    stream = r.clone()
    awq.linear_fused(x, pw, residual=stream, y=stream)
    assert torch.equal(apart, stream)


@pytest.mark.parametrize("M", [1, 6, 13, 61, 400])
def test_same_bits_again_on_another_stream_and_in_a_graph(M):
    awq = G.lib()
    N, K = 1040, 2048
    pw, _ = H.packed_layer(awq, N, K, 128, True, 4)
    x, b = G.dev_f16(workloads.activations(M, K, cfg=11, layer=4)), G.dev_f16(H.halves(N, 4))
    first = awq.linear_fused(x, pw, b, "silu", True)
    assert torch.equal(first, awq.linear_fused(x, pw, b, "silu", True))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = awq.linear_fused(x, pw, b, "silu", True)
        y = torch.empty_like(first)
        graph = torch.cuda.CUDAGraph()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            awq.linear_fused(x, pw, b, "silu", True, y=y)
    side.synchronize()
    assert torch.equal(first, there)
    for _ in range(4):
        y.zero_()
        graph.replay()
        assert torch.equal(awq.linear_fused(x, pw, b, "silu", True), first)
        torch.cuda.synchronize()
        assert torch.equal(y, first)


@pytest.mark.parametrize("M", [3, 12, 50, 200])
def test_a_row_that_is_not_finite_stays_alone(M):
    """An infinity or NaN in one token's activations reaches no other token."""
    awq = G.lib()
    pw, wdq = H.packed_layer(awq, 136, 288, 32, True, 6)
    X = workloads.activations(M, 288, cfg=11, layer=6)
    bad = X.copy()
    bad[1, 5], bad[M - 1, 200] = np.inf, np.nan
    y = G.host_f16(awq.linear_fused(G.dev_f16(bad), pw, None, "relu"))
    assert not np.isfinite(y[1]).any() or not np.isfinite(y[1]).all()
    assert np.isnan(y[M - 1]).all()
    keep = np.array([i for i in range(M) if i not in (1, M - 1)])
    ref, bound = F.linear_fused(X[keep], wdq, None, "relu")
    H.check(y[keep], ref, bound, f"beside a bad row, M={M}")


def test_offsets_past_32_bits():
    """Rows of x and y more than 2^32 bytes from the first one."""
    awq = G.lib()
    M, N, K, ld = 70000, 8, 64, 32768  # 70000 rows * 64 KiB = 4.6 GB each
    pw, wdq = H.packed_layer(awq, N, K, 32, True, 2)
    x = torch.empty((M, ld), dtype=torch.float16, device="cuda")
    X = workloads.activations(M, K, cfg=11, layer=2)
    x[:, :K] = G.dev_f16(X)
    y = torch.empty((M, ld), dtype=torch.float16, device="cuda")
    awq.linear_fused(x[:, :K], pw, y=y[:, :N])
    pick = np.r_[0:40, 32740:32800, 65510:65560, M - 300:M]
    ref, bound = F.linear_fused(X[pick], wdq)
    H.check(G.host_f16(y[:, :N].contiguous())[pick], ref, bound, "far rows")


def test_mlp_is_its_two_layers():
    awq = G.lib()
    K, Fw = 256, 320
    gu, wgu = H.packed_layer(awq, 2 * Fw, K, 64, True, 21)
    dn, wdn = H.packed_layer(awq, K, Fw, 32, True, 22)
    for M in (1, 7, 33):
        X, r = workloads.activations(M, K, cfg=11, layer=M), H.halves((M, K), M)
        x = G.dev_f16(X)
        y = awq.mlp(x, gu, dn, residual=G.dev_f16(r))
        h = awq.linear_fused(x, gu, activation="silu", gated=True)
        assert torch.equal(y, awq.linear_fused(h, dn, residual=G.dev_f16(r)))
        H.check(G.host_f16(y), *F.linear_fused(G.host_f16(h), wdn, residual=r), f"mlp M={M}")


def test_leading_dimensions():
    awq = G.lib()
    pw, _ = H.packed_layer(awq, 64, 128, 32, True, 1)
    x = G.dev_f16(workloads.activations(6, 128, cfg=11, layer=1))
    r = G.dev_f16(H.halves((6, 64), 1))
    y = awq.linear_fused(x.reshape(2, 3, 128), pw, residual=r.reshape(2, 3, 64))
    assert y.shape == (2, 3, 64) and torch.equal(y.reshape(6, 64), awq.linear_fused(x, pw, residual=r))


def test_no_activation_matches_the_plain_layer_closely():
    """Without an epilogue the fused layer is the plain one: both within the contract of the exact product."""
    awq = G.lib()
    pw, wdq = H.packed_layer(awq, 512, 1024, 128, True, 9)
    for M in (1, 5, 20, 90):
        X = workloads.activations(M, 1024, cfg=11, layer=9)
        ref, bound = F.linear_fused(X, wdq)
        H.check(G.host_f16(awq.linear_fused(G.dev_f16(X), pw)), ref, bound, f"fused M={M}")
        H.check(G.host_f16(awq.linear(G.dev_f16(X), pw)), ref, bound, f"plain M={M}")
