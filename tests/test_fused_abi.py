"""The fused layer, router and expert products refuse what they cannot take, on the host and before any launch (no GPU
needed: every call below fails validation, so no pointer is dereferenced); and the oracle's own forms agree with
hand-worked values and with a second statement of them."""
from __future__ import annotations

import math
import os

import numpy as np
import pytest

from oracle import fused_oracle as F

awq = pytest.importorskip("bit_weight_only_awq_amd")
torch = pytest.importorskip("torch")

A = 0x7F0000000000
B, C, D, E_, Y, W, R = (A + i * 0x100000 for i in range(1, 8))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(awq.LIB_PATH):
        pytest.fail(f"{awq.LIB_PATH} not built; run python -m bit_weight_only_awq_amd.build")
    return awq.load_library()


def test_strerror_names_the_option_error(lib):
    assert "option" in awq.awq_strerror(awq.AWQ_ERR_OPTION)


def test_linear_fused_refusals(lib):
    def call(**kw):
        a = dict(x=A, ldx=128, qw=B, sc=C, qz=D, bias=E_, act=0, gated=0, res=R, ldr=16, y=Y, ldy=16, M=4, N=16, K=128,
                 g=32, zp=1, ws=W, wsb=1 << 40)
        a.update(kw)
        return lib.awq_linear_fused(*(a[k] or None if k in ("x", "qw", "sc", "qz", "bias", "res", "y", "ws") else a[k]
                                      for k in ("x", "ldx", "qw", "sc", "qz", "bias", "act", "gated", "res", "ldr", "y",
                                                "ldy", "M", "N", "K", "g", "zp", "ws", "wsb")), None)

    for kw in (dict(M=0), dict(M=-1), dict(M=(1 << 24) + 1), dict(N=0), dict(N=12), dict(K=0), dict(N=1 << 22),
               dict(ldx=120), dict(ldx=132), dict(ldy=8), dict(ldy=18), dict(ldr=8), dict(gated=1, N=24),
               dict(gated=1, ldy=4), dict(ldx=-128)):
        assert call(**kw) == awq.AWQ_ERR_SHAPE, kw
    for kw in (dict(g=48), dict(g=0), dict(K=96, g=64)):
        assert call(**kw) == awq.AWQ_ERR_GROUP, kw
    for kw in (dict(act=-1), dict(act=5)):
        assert call(**kw) == awq.AWQ_ERR_OPTION, kw
    for name in ("x", "qw", "sc", "qz", "y"):
        assert call(**{name: 0}) == awq.AWQ_ERR_NULL, name
    for name, at in (("x", A), ("qw", B), ("sc", C), ("qz", D), ("y", Y), ("bias", E_), ("res", R)):
        assert call(**{name: at + 8}) == awq.AWQ_ERR_ALIGN, name
    need = lib.awq_linear_fused_workspace_bytes(16, 4096, 4096, 128, 0)
    if need:
        big = dict(M=16, N=4096, K=4096, g=128, ldx=4096, ldy=4096, ldr=4096)
        assert call(**big, wsb=need - 1) == awq.AWQ_ERR_WORKSPACE
        assert call(**big, ws=0) == awq.AWQ_ERR_NULL
        assert call(**big, ws=W + 8) == awq.AWQ_ERR_ALIGN
    for bad in ((0, 16, 128, 32, 0), (4, 12, 128, 32, 0), (4, 24, 128, 32, 1), (4, 16, 128, 48, 0)):
        assert lib.awq_linear_fused_workspace_bytes(*bad) == 0, bad


def test_route_refusals(lib):
    def call(**kw):
        a = dict(x=A, ld=8, f32=1, T=4, E=8, k=2, ids=B, w=C, off=D, rows=E_, pos=Y, ws=W, wsb=1 << 30)
        a.update(kw)
        return lib.awq_route_experts(a["x"] or None, a["ld"], a["f32"], a["T"], a["E"], a["k"], 1, a["ids"] or None,
                                     a["w"] or None, a["off"] or None, a["rows"] or None, a["pos"] or None,
                                     a["ws"] or None, a["wsb"], None)

    for kw in (dict(T=0), dict(E=0), dict(E=1025, ld=1025), dict(ld=7), dict(T=(1 << 24) + 1), dict(T=1 << 23, k=3)):
        assert call(**kw) == awq.AWQ_ERR_SHAPE, kw
    for kw in (dict(k=0), dict(k=9), dict(E=100, ld=100, k=65)):
        assert call(**kw) == awq.AWQ_ERR_OPTION, kw
    for name in ("x", "ids", "w", "off", "rows", "pos"):
        assert call(**{name: 0}) == awq.AWQ_ERR_NULL, name
        assert call(**{name: dict(x=A, ids=B, w=C, off=D, rows=E_, pos=Y)[name] + 4}) == awq.AWQ_ERR_ALIGN, name
    need = lib.awq_route_experts_workspace_bytes(100000, 64)
    assert need > 0 and lib.awq_route_experts_workspace_bytes(1, 64) == 0
    assert call(T=100000, E=64, ld=64, wsb=need - 1) == awq.AWQ_ERR_WORKSPACE
    assert call(T=100000, E=64, ld=64, ws=0) == awq.AWQ_ERR_NULL
    assert lib.awq_route_experts_workspace_bytes(0, 8) == 0 and lib.awq_route_experts_workspace_bytes(9, 2000) == 0


def test_expert_products_refusals(lib):
    def rows(**kw):
        a = dict(x=A, ldx=128, xr=4, rows=B, spr=2, off=C, R=8, E=4, qw=D, sc=E_, qz=Y, bias=W, act=2, gated=1, y=R,
                 ldy=8, N=16, K=128, g=32, zp=1)
        a.update(kw)
        return lib.awq_linear_experts(a["x"] or None, a["ldx"], a["xr"], a["rows"] or None, a["spr"], a["off"] or None,
                                      a["R"], a["E"], a["qw"] or None, a["sc"] or None, a["qz"] or None,
                                      a["bias"] or None, a["act"], a["gated"], a["y"] or None, a["ldy"], a["N"],
                                      a["K"], a["g"], a["zp"], None, 0, None)

    for kw in (dict(R=0), dict(E=0), dict(E=1025), dict(xr=0), dict(rows=0), dict(N=8), dict(ldy=4), dict(ldx=64)):
        assert rows(**kw) == awq.AWQ_ERR_SHAPE, kw
    assert rows(spr=0) == awq.AWQ_ERR_OPTION and rows(act=9) == awq.AWQ_ERR_OPTION
    assert rows(g=100) == awq.AWQ_ERR_GROUP
    for name in ("x", "off", "qw", "sc", "qz", "y"):
        assert rows(**{name: 0}) == awq.AWQ_ERR_NULL, name
    for name, at in (("rows", B), ("off", C), ("bias", W), ("y", R)):
        assert rows(**{name: at + 2}) == awq.AWQ_ERR_ALIGN, name

    def combine(**kw):
        a = dict(x=A, ldx=128, off=B, pos=C, w=D, T=4, k=2, E=4, qw=E_, sc=Y, qz=W, bias=0, res=R, ldr=16,
                 y=R + 0x1000, ldy=16, N=16, K=128, g=32, ws=A + 0x900000, wsb=1 << 40)
        a.update(kw)
        return lib.awq_combine_experts(a["x"] or None, a["ldx"], a["off"] or None, a["pos"] or None, a["w"] or None,
                                       a["T"], a["k"], a["E"], a["qw"] or None, a["sc"] or None, a["qz"] or None,
                                       a["bias"] or None, a["res"] or None, a["ldr"], a["y"] or None, a["ldy"], a["N"],
                                       a["K"], a["g"], 1, a["ws"] or None, a["wsb"], None)

    for kw in (dict(T=0), dict(E=0), dict(ldr=8), dict(T=1 << 24, k=4), dict(N=20)):
        assert combine(**kw) == awq.AWQ_ERR_SHAPE, kw
    assert combine(k=0) == awq.AWQ_ERR_OPTION and combine(k=5) == awq.AWQ_ERR_OPTION
    for name in ("off", "pos", "w"):
        assert combine(**{name: 0}) == awq.AWQ_ERR_NULL, name
    need = lib.awq_combine_experts_workspace_bytes(4, 2, 4, 16, 128, 32)
    if need:
        assert combine(wsb=need - 1) == awq.AWQ_ERR_WORKSPACE and combine(ws=0) == awq.AWQ_ERR_NULL
    for bad in ((0, 2, 4, 16, 128, 32), (4, 2, 0, 16, 128, 32), (4, 2, 4, 20, 128, 32)):
        assert lib.awq_combine_experts_workspace_bytes(*bad) == 0, bad


def test_binding_refusals():
    x = torch.zeros((2, 128), dtype=torch.float16)
    pw = awq.PackedWeight(torch.zeros((16, 16), dtype=torch.int32), torch.zeros((2, 4, 8), dtype=torch.float16),
                          torch.zeros((2, 4), dtype=torch.int32), 16, 128, 32, True)
    for bad in (x, x.float(), x[:, :64]):  # on the host, another type, another width
        with pytest.raises(ValueError):
            awq.linear_fused(bad, pw)
    with pytest.raises(ValueError):
        awq.route_experts(x.double(), 1)
    with pytest.raises(ValueError):
        awq.route_experts(x, 1)  # on the host
    with pytest.raises(ValueError):
        awq.pack_experts(x)
    with pytest.raises(ValueError, match="activation"):
        awq._activation("tanh")
    with pytest.raises(ValueError, match="bias"):
        awq._flat(torch.zeros(8, dtype=torch.float16), (16,), torch.float16, "bias")


def test_oracle_route_by_hand():
    inf, nan = math.inf, math.nan
    v = np.array([[0.0, 1.0, 1.0, -inf], [-inf, nan, -inf, -inf], [inf, 2.0, inf, nan]], np.float32)
    ids, w, offsets, rows, positions = F.route(v, 2, True)
    assert ids.tolist() == [[1, 2], [-1, -1], [0, 2]]
    assert np.allclose(w, [[0.5, 0.5], [0, 0], [0.5, 0.5]])
    assert offsets.tolist() == [0, 1, 2, 4, 4]
    assert rows.tolist() == [4, 0, 1, 5, -1, -1]
    assert positions.tolist() == [[1, 2], [-1, -1], [0, 3]]
    _, w, *_ = F.route(v[:1], 2, False)
    assert np.allclose(w, np.e / (1 + 2 * np.e))


def test_oracle_activations():
    v = np.linspace(-6, 6, 41)
    assert np.allclose(F.activation(v, "silu"), v * 0.5 * (1 + np.tanh(v / 2)))
    assert np.max(np.abs(F.activation(v, "gelu") - F.activation(v, "gelu_tanh"))) < 1e-3
    for act in ("silu", "gelu", "gelu_tanh", "relu", "none"):  # the slope the bounds rest on
        f = np.linspace(-12, 12, 24001)
        assert np.max(np.abs(np.diff(F.activation(f, act)) / np.diff(f))) <= F.SLOPE


def test_oracle_combine_is_a_dense_mixture():
    """The sorted, ragged form equals every expert on every token times its (mostly zero) weight."""
    rng = np.random.default_rng(1)
    T, E, k, N, K = 9, 5, 2, 8, 16
    W = [rng.standard_normal((N, K)) for _ in range(E)]
    X = rng.standard_normal((T, K)).astype(np.float16)
    ids, w, offsets, rows, positions = F.route(rng.standard_normal((T, E)), k, True)
    y, _ = F.combine_experts(X[rows // k], W, offsets, positions, w)
    dense = np.zeros((T, N))
    for t in range(T):
        for j in range(k):
            dense[t] += w[t, j] * (W[ids[t, j]] @ X[t].astype(np.float64))
    assert np.allclose(y, dense)
