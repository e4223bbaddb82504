"""Products in two launches (partial sums, then their sum) called by two host threads on one stream: the first launches of
both may be enqueued before the second of either, so their partial sums must lie in different memory."""
from __future__ import annotations

import threading

import pytest

awq = pytest.importorskip("bit_weight_only_awq_amd")
torch = pytest.importorskip("torch")

NEED = 1 << 21


def test_concurrent_calls_have_workspaces_of_their_own(monkeypatch):
    kept = torch.zeros(NEED, dtype=torch.uint8)  # what a buffer kept for the stream would be
    monkeypatch.setattr(awq, "gemm_workspace", lambda nbytes, device=None, stream=None: kept)
    both, used, like = threading.Barrier(2), [], torch.zeros(1)

    def call(address, nbytes):
        if not address or nbytes < NEED:
            return awq.AWQ_ERR_WORKSPACE
        both.wait(20)  # both calls hold their workspaces
        used.append(address)
        both.wait(20)
        return awq.AWQ_OK

    threads = [threading.Thread(target=awq._with_workspace, args=(call, lambda: NEED, "product", None, like))
               for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(used) == 2 and abs(used[0] - used[1]) >= NEED


def test_a_given_workspace_is_the_one_used():
    ws, seen = torch.zeros(NEED, dtype=torch.uint8), []

    def call(address, nbytes):
        seen.append((address, nbytes))
        return awq.AWQ_OK if nbytes >= NEED else awq.AWQ_ERR_WORKSPACE

    def ptr(t):
        return None if t is None else t.data_ptr()

    with pytest.MonkeyPatch.context() as m:
        m.setattr(awq, "_ptr", ptr)
        awq._with_workspace(call, lambda: NEED, "product", ws, ws)
        assert seen == [(ws.data_ptr(), NEED)]
        with pytest.raises(awq.AwqError) as e:
            awq._with_workspace(call, lambda: NEED, "product", ws[:16], ws)
    assert e.value.status == awq.AWQ_ERR_WORKSPACE
