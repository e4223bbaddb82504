"""Calls with ever larger batches keep no memory behind them: only what a caller or a captured graph still holds."""
from __future__ import annotations

import pytest

from tests import _gpu as G

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def test_rising_batches_leave_no_workspaces_behind():
    awq = G.lib()
    E, k, N, K = 4, 2, 4096, 64
    gen = torch.Generator(device="cuda").manual_seed(3)
    pe = awq.pack_experts((torch.randn((E, N, K), generator=gen, device="cuda") / 8).half(), 64, True)
    pw = awq.pack((torch.randn((4096, 11008), generator=gen, device="cuda") / 100).half())
    lib = awq.load_library()
    batches = range(400, 600, 8)
    largest = max(lib.awq_combine_experts_workspace_bytes(T, k, E, N, K, 64) for T in batches)
    assert largest > 10 << 20
    assert len({lib.awq_linear_fused_workspace_bytes(M, 4096, 11008, 128, 0) for M in range(9, 17)}) == 8
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        logits = torch.randn((600, E), generator=gen, device="cuda")
        h = torch.randn((1200, K), generator=gen, device="cuda").half()
        x = torch.randn((16, 11008), generator=gen, device="cuda").half()
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        for T in batches:
            awq.combine_experts(h[:T * k], pe, awq.route_experts(logits[:T], k))
        for M in range(9, 17):
            awq.linear_fused(x[:M], pw)
        torch.cuda.synchronize()
        assert torch.cuda.memory_allocated() - before <= largest


def test_first_call_of_a_split_product_in_a_graph():
    """No earlier eager call on the capturing stream is needed, and replays repeat the eager result."""
    awq = G.lib()
    gen = torch.Generator(device="cuda").manual_seed(4)
    pw = awq.pack((torch.randn((4096, 11008), generator=gen, device="cuda") / 100).half())
    x = torch.randn((13, 11008), generator=gen, device="cuda").half()
    assert awq.load_library().awq_linear_fused_workspace_bytes(13, 4096, 11008, 128, 0) > 0
    want = awq.linear_fused(x, pw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y = awq.linear_fused(x, pw)
    for _ in range(4):
        y.zero_()
        graph.replay()
        assert torch.equal(awq.linear_fused(x, pw), want)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
