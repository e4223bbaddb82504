"""pack_experts is pack expert by expert, also where an expert's zero points do not fill whole 16-byte units, and where
the experts' rows together exceed what one call packs."""
from __future__ import annotations

import pytest

import workloads
from tests import _gpu as G

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def weights(E, N, K):
    return torch.stack([G.dev_f16(workloads.weight(N, K, cfg=12, layer=e)) for e in range(E)])


def same_as_pack(awq, pe, W, g, zp):
    assert (pe.E, pe.N, pe.K, pe.group_size, pe.zero_point) == (*W.shape, g, zp)
    for e in range(W.shape[0]):
        one = awq.pack(W[e].contiguous(), g, zp)
        assert torch.equal(pe.qweight[e], one.qweight) and torch.equal(pe.scales[e], one.scales), e
        assert pe.qzeros is None if not zp else torch.equal(pe.qzeros[e], one.qzeros), e


# (N / 8)(K / g): 5, 27, 9, 2 and 4 words of zero points for each expert
@pytest.mark.parametrize("N,K,g", [(40, 128, 128), (72, 96, 32), (24, 768, 256), (16, 64, 64), (32, 64, 64)])
@pytest.mark.parametrize("E", [1, 2, 7])
@pytest.mark.parametrize("zp", [True, False])
def test_zero_points_of_any_number_of_words(E, N, K, g, zp):
    awq = G.lib()
    W = weights(E, N, K)
    same_as_pack(awq, awq.pack_experts(W, g, zp), W, g, zp)
    same_as_pack(awq, awq.pack_experts(list(W), g, zp), W, g, zp)


@pytest.mark.parametrize("rows", [40, 100, 130, 170, 1 << 20])
def test_more_rows_than_one_call_packs(monkeypatch, rows):
    awq = G.lib()
    monkeypatch.setattr(awq, "_PACK_ROWS", rows)
    W = weights(9, 40, 128)
    for zp in (True, False):
        same_as_pack(awq, awq.pack_experts(W, 128, zp), W, 128, zp)


def test_refusals():
    awq = G.lib()
    for N, K, g, status in ((4, 64, 32, awq.AWQ_ERR_SHAPE), (12, 64, 32, awq.AWQ_ERR_SHAPE),
                            (16, 96, 64, awq.AWQ_ERR_GROUP), (16, 64, 48, awq.AWQ_ERR_GROUP)):
        with pytest.raises(awq.AwqError) as e:
            awq.pack_experts(torch.zeros((4, N, K), dtype=torch.float16, device="cuda"), g)
        assert e.value.status == status
