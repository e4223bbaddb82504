"""The epilogue alone: activations on pre-activations that are exact (x is zero, the bias holds the values), so that the
bounds are those of the fp32 epilogue and the one rounding, in every kernel that applies it."""
from __future__ import annotations

import math

import numpy as np
import pytest

from oracle import fused_oracle as F
from tests import _gpu as G

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

V = np.unique(np.r_[np.arange(-768, 769) / 64.0, np.linspace(-6, -3, 87)].astype(np.float16)).astype(np.float64)
V = np.r_[V, np.zeros(-len(V) % 16)]


def exact(v, act):
    """The definition in 64 bits; gelu through erfc, which does not cancel."""
    if act == "gelu":
        return np.array([0.5 * x * math.erfc(-x / math.sqrt(2.0)) for x in v])
    if act == "gelu_tanh":  # 0.5 (1 + tanh u) = 1 / (1 + exp(-2 u))
        return v / (1.0 + np.exp(-2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    return F.activation(v, act)


def relative(v, act):
    """The relative error that the fp32 form is allowed, in units of 2^-24.  silu: the exponent's argument v log2 e
    carries the rounding of the constant and of the product (2 |v|), the exponential and the reciprocal 2 each, the sum
    and the product 1 each.  gelu (tanh form): the same with u = 2 sqrt(2 / pi) (v + 0.044715 v^3), itself off by five
    roundings.  gelu: the argument t = v / sqrt 2 is off by two roundings, which erfc (and so the result) magnifies by
    t erfc'(t) / erfc(t) < 2 t^2 + 2 = v^2 + 2; erfc itself 32 (16 units in the last place); three products."""
    a = np.abs(v)
    if act == "silu":
        return 2 * a + 8
    if act == "gelu_tanh":
        u = 2.0 * math.sqrt(2.0 / math.pi) * (a + 0.044715 * a ** 3)
        return 7 * u + 8
    return 2 * (a * a + 2) + 35


# one token, a few, 16-row tiles with and without a split, 32-row tiles in groups of 32, matrix-core tiles
@pytest.mark.parametrize("M,K,g", [(1, 64, 64), (4, 64, 64), (13, 11008, 128), (16, 64, 64), (40, 64, 32), (300, 64, 64)])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gated", [False, True])
def test_activations_on_exact_values(M, K, g, act, gated):
    awq = G.lib()
    up = np.where(np.arange(len(V)) % 2 == 0, 100.0, -300.0)
    bias = np.r_[V, up] if gated else V
    N = len(bias)
    gen = torch.Generator(device="cuda").manual_seed(1)
    pw = awq.pack(torch.randn((N, K), generator=gen, device="cuda").half(), g, True)
    x = torch.zeros((M, K), dtype=torch.float16, device="cuda")
    y = G.host_f16(awq.linear_fused(x, pw, G.dev_f16(bias), act, gated)).astype(np.float64)
    ref = exact(V, act) * (up if gated else 1.0)
    bound = (relative(V, act) + 1) * 2.0 ** -24 * np.abs(ref) + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25
    off = np.abs(y - ref) / bound
    m, i = np.unravel_index(np.argmax(off), off.shape)
    assert off[m, i] <= 1.0, f"{act} gated={gated} M={M}: at {V[i]}: {y[m, i]} for {ref[i]}"
