"""Products that split K refuse a workspace that is too small, missing or misaligned, before any launch (no GPU needed:
every call below fails validation)."""
from __future__ import annotations

import os

import pytest

awq = pytest.importorskip("bit_weight_only_awq_amd")

A = 0x7F0000000000
X, Q, S, Z, Y, W, OFF, POS, WT, ROWS = (A + i * 0x10000000 for i in range(10))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(awq.LIB_PATH):
        pytest.fail(f"{awq.LIB_PATH} not built; run python -m bit_weight_only_awq_amd.build")
    return awq.load_library()


def refuses(call, need):
    assert need > 0
    for ws, nbytes, status in ((W, need - 1, awq.AWQ_ERR_WORKSPACE), (W, 0, awq.AWQ_ERR_WORKSPACE),
                               (None, 0, awq.AWQ_ERR_WORKSPACE), (None, need, awq.AWQ_ERR_NULL),
                               (W + 8, need, awq.AWQ_ERR_ALIGN)):
        assert call(ws, nbytes) == status, (ws, nbytes)


@pytest.mark.parametrize("M,N,K,gated", [(13, 4096, 11008, 0), (16, 2048, 11008, 1), (100, 4096, 4096, 0)])
def test_linear_fused(lib, M, N, K, gated):
    refuses(lambda ws, n: lib.awq_linear_fused(X, K, Q, S, Z, None, 0, gated, None, 0, Y, N, M, N, K, 128, 1, ws, n, None),
            lib.awq_linear_fused_workspace_bytes(M, N, K, 128, gated))


@pytest.mark.parametrize("T,k,E,N,K", [(20, 2, 6, 144, 7168), (100, 2, 6, 144, 11008)])
def test_linear_experts(lib, T, k, E, N, K):
    for gated in (0, 1):
        refuses(lambda ws, n: lib.awq_linear_experts(X, K, T, ROWS, k, OFF, T * k, E, Q, S, Z, None, 0, gated, Y, N, N, K,
                                                     64, 1, ws, n, None),
                lib.awq_linear_experts_workspace_bytes(T * k, E, N, K, 64, gated))


@pytest.mark.parametrize("T,k,E,N,K", [(4, 2, 4, 16, 128), (20, 2, 6, 144, 7168), (1000, 2, 8, 4096, 11008)])
def test_combine_experts(lib, T, k, E, N, K):
    refuses(lambda ws, n: lib.awq_combine_experts(X, K, OFF, POS, WT, T, k, E, Q, S, Z, None, None, 0, Y, N, N, K, 128, 1,
                                                  ws, n, None),
            lib.awq_combine_experts_workspace_bytes(T, k, E, N, K, 128))
