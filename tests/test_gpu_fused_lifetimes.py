"""Copies that linear_fused makes of its arguments are held until the kernels that read them are enqueued."""
from __future__ import annotations

import pytest

from tests import _gpu as G

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


class Watched:
    """The library, with the memory in use noted at each call of the fused layer."""

    def __init__(self, lib):
        self.lib, self.seen = lib, []

    def __getattr__(self, name):
        return getattr(self.lib, name)

    def awq_linear_fused(self, *args):
        self.seen.append(torch.cuda.memory_allocated())
        return self.lib.awq_linear_fused(*args)


def test_a_residual_copied_for_its_layout_lives_through_the_call(monkeypatch):
    """A residual of three dimensions with swapped strides is copied first: the copy is held until the kernels that read
    it are enqueued, so that no memory of the same call (partial sums) takes its place."""
    awq = G.lib()
    M, N, K = 300, 4096, 11008
    gen = torch.Generator(device="cuda").manual_seed(5)
    pw = awq.pack((torch.randn((N, K), generator=gen, device="cuda") / 100).half())
    lib = awq.load_library()
    need = lib.awq_linear_fused_workspace_bytes(M, N, K, 128, 0)
    assert need > 0
    x = torch.randn((2, M // 2, K), generator=gen, device="cuda").half()
    residual = torch.randn((M // 2, 2, N), generator=gen, device="cuda").half().transpose(0, 1)
    want = awq.linear_fused(x, pw, residual=residual.contiguous())
    y = torch.empty((M, N), dtype=torch.float16, device="cuda")
    watched = Watched(lib)
    monkeypatch.setattr(awq, "_lib", watched)
    before = torch.cuda.memory_allocated()
    awq.linear_fused(x, pw, residual=residual, y=y)
    assert torch.equal(y.view(2, M // 2, N), want)
    assert watched.seen[-1] >= before + residual.numel() * 2 + need
