"""A slice of the experts: offsets that begin above zero, as a process that holds some of the experts takes them from the
whole route.  Only the slice's rows are computed and added up, in every kernel; nothing else is written, and nothing is
read from a workspace that no kernel wrote."""
from __future__ import annotations

import numpy as np
import pytest

import workloads
from oracle import fused_oracle as F
from tests import _fused as H
from tests import _gpu as G
from tests.test_gpu_experts import device_route, logits_of

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

E, LO, HI = 12, 3, 9


def stale(nbytes):
    """A workspace whose every float is NaN (None where none is needed)."""
    return torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda") if nbytes else None


# one row for each expert or fewer, 4-row tiles, 16- and 32-row tiles (K split and not), matrix-core tiles
@pytest.mark.parametrize("T,N,K", [(1, 144, 256), (3, 144, 256), (5, 144, 256), (9, 144, 256), (20, 144, 7168),
                                   (60, 144, 256), (100, 144, 11008), (170, 144, 256), (500, 144, 256),
                                   (1000, 2064, 2048)])
def test_only_the_slice_is_computed(T, N, K):
    awq = G.lib()
    k = 1 if T == 3 else 2
    logits = logits_of(T, E, 21)
    if T <= 3:  # slots on both sides of the slice and in it
        logits[0, [0, 5]] = 9.0
    ids, weights, offsets, rows, positions = F.route(logits, k, True)
    pe, wdq = H.packed_experts(awq, HI - LO, N, K, 64, True, T)
    route = device_route(awq, (ids, weights, offsets[LO:HI + 1], rows, positions))
    lo, hi = int(offsets[LO]), int(offsets[HI])
    assert T <= 3 or 0 < lo < hi < T * k
    X, b = workloads.activations(T, K, cfg=12, layer=T), H.halves((HI - LO, N), T)
    lib = awq.load_library()
    for gated in (False, True):
        y = torch.full((T * k, N // 2 if gated else N), 55.0, dtype=torch.float16, device="cuda")
        awq.linear_experts(G.dev_f16(X), pe, route, G.dev_f16(b), "silu", gated, y=y, workspace=stale(
            lib.awq_linear_experts_workspace_bytes(T * k, HI - LO, N, K, 64, int(gated))))
        got = G.host_f16(y)
        assert np.all(got[:lo] == 55.0) and np.all(got[hi:] == 55.0), f"T={T}: a row of no expert was written"
        if hi > lo:
            ref = F.linear_experts(X, wdq, offsets[LO:HI + 1], rows, k, b, "silu", gated)
            H.check(got[lo:hi], *ref, f"slice of experts, rows, T={T} gated={gated}")
    h, r = workloads.activations(T * k, K, cfg=12, layer=T + 1), H.halves((T, N), T + 2)
    inside = np.where((positions >= lo) & (positions < hi), positions, -1)
    ref = F.combine_experts(h, wdq, offsets[LO:HI + 1], inside, weights.astype(np.float32), b, r)
    y = awq.combine_experts(G.dev_f16(h), pe, route, G.dev_f16(b), G.dev_f16(r), workspace=stale(
        lib.awq_combine_experts_workspace_bytes(T, k, HI - LO, N, K, 64)))
    H.check(G.host_f16(y), *ref, f"slice of experts, combined, T={T}")


@pytest.mark.parametrize("T", [1, 30, 500])
def test_slices_of_one_route_add_up(T):
    """Views of the route's offsets as they are: the parts of three processes, each on the residual stream of the one
    before, against all experts at once."""
    awq = G.lib()
    N, K, k = 80, 128, 2
    logits = logits_of(T, E, 22)
    pe, wdq = H.packed_experts(awq, E, N, K, 32, True, 5)
    route = awq.route_experts(torch.from_numpy(logits).cuda(), k)
    h = workloads.activations(T * k, K, cfg=12, layer=5)
    hd = G.dev_f16(h)
    _, weights, offsets, _, positions = F.route(logits, k, True)
    y, total = np.zeros((T, N)), np.zeros((T, N))
    for lo, hi in ((0, 5), (5, 7), (7, 12)):
        part = awq.PackedExperts(pe.qweight[lo:hi].clone(), pe.scales[lo:hi].clone(), pe.qzeros[lo:hi].clone(), hi - lo,
                                 N, K, 32, True)
        got = awq.combine_experts(hd, part, route._replace(offsets=route.offsets[lo:hi + 1]))
        inside = np.where((positions >= offsets[lo]) & (positions < offsets[hi]), positions, -1)
        ref, bound = F.combine_experts(h, wdq[lo:hi], offsets[lo:hi + 1], inside, weights.astype(np.float32))
        H.check(G.host_f16(got), ref, bound, f"experts {lo} .. {hi - 1}, T={T}")
        y += G.host_f16(got).astype(np.float64)
        total += bound
    ref, bound = F.combine_experts(h, wdq, offsets, positions, weights.astype(np.float32))
    assert np.all(np.abs(y - ref) <= total + bound)
