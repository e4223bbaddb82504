"""A decoder block's attention as it is used: the fused q/k/v layer, tokens appended, attention over the cache (all
pages, a shared prefix, chosen pages) and the output layer, over several steps, against fp64 of the same block."""
from __future__ import annotations

import numpy as np
import pytest

from tests import _gpu as G
from tests._fused import halves, packed_layer

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

K, HQ, HKV, D, S = 512, 8, 2, 64, 16


def reference(x, wqkv, wo, past, freq, residual):
    """One sequence's block in fp64, the cache's keys and values rounded to fp16 as they are stored."""
    n, at = len(x), len(past[0])
    rows = (x.astype(np.float64) @ wqkv.T).astype(np.float16).astype(np.float64).reshape(n, HQ + 2 * HKV, D)
    angle = (at + np.arange(n))[:, None] * freq.astype(np.float64)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    a, b = rows[:, :HQ + HKV, :D // 2].copy(), rows[:, :HQ + HKV, D // 2:].copy()
    rows[:, :HQ + HKV] = np.concatenate([a * c - b * s, b * c + a * s], 2)
    rows = rows.astype(np.float16)
    k = past[0] = np.concatenate([past[0], rows[:, HQ:HQ + HKV]])
    v = past[1] = np.concatenate([past[1], rows[:, HQ + HKV:]])
    y = np.zeros((n, HQ, D))
    for i in range(n):
        for h in range(HQ):
            score = k[:at + i + 1, h * HKV // HQ].astype(np.float64) @ rows[i, h].astype(np.float64) * D ** -0.5
            w = np.exp(score - score.max())
            y[i, h] = w @ v[:at + i + 1, h * HKV // HQ].astype(np.float64) / w.sum()
    return y.reshape(n, -1) @ wo.T + residual.astype(np.float64)


@pytest.mark.parametrize("mode", ["all", "shared", "pages"])
def test_block_over_steps(mode):
    awq = G.lib()
    pw, wqkv = packed_layer(awq, (HQ + 2 * HKV) * D, K, 128, True, 3)
    po, wo = packed_layer(awq, K, HQ * D, 64, False, 4)
    freq = (10000.0 ** (-np.arange(0, D, 2) / D)).astype(np.float32)
    B, prompt = 3, 64
    cache = awq.kv_cache(40, HKV, D, S, bounds=True)
    cache.k.fill_(float("nan"))
    cache.v.fill_(float("nan"))
    tables = np.zeros((B, 12), np.int32)
    order = np.random.default_rng(0).permutation(40)
    tables[:, :prompt // S] = order[:prompt // S]
    tables[:, prompt // S:] = order[prompt // S:prompt // S + B * 8].reshape(B, 8)
    i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    past = [[np.zeros((0, HKV, D), np.float16)] * 2]
    past[0] = list(past[0])

    def check(y, ref, what):
        y = y.cpu().numpy().astype(np.float64)
        # every stage rounds to fp16 (q/k/v rows, their rotation, weights, the attention's result, the output): five
        # roundings of 2^-11 / sqrt 3 each in the mean square, 6.3e-4 in all; scores of a few units turn 2^-11 of them
        # into as much of a weight again: 2e-3 leaves a factor of two
        assert np.linalg.norm(y - ref) <= 2e-3 * np.linalg.norm(ref), what

    # the common prompt, once, as one sequence
    x, r = halves((prompt, K), 1), halves((prompt, K), 2)
    y = awq.attention(dev(x), pw, po, cache, awq.Sequences(i32([0, prompt]), i32([prompt]), i32(tables[:1])), dev(freq),
                      residual=dev(r))
    check(y, reference(x, wqkv, wo, past[0], freq, r), "prompt")
    past = [list(past[0]) for _ in range(B)]
    lengths = np.full(B, prompt)
    for step, new in enumerate(([20, 5, 1], [1, 1, 1], [1, 1, 1], [2, 1, 3], [1, 1, 1])):
        T = sum(new)
        x, r = halves((T, K), 10 + step), halves((T, K), 30 + step)
        lengths = lengths + new
        offsets = np.concatenate([[0], np.cumsum(new)])
        seqs = awq.Sequences(i32(offsets), i32(lengths), i32(tables))
        kw = {"shared": prompt} if mode == "shared" else {"pages": 12} if mode == "pages" else {}
        y = awq.attention(dev(x), pw, po, cache, seqs, dev(freq), residual=dev(r), **kw)
        ref = np.concatenate([reference(x[offsets[b]:offsets[b + 1]], wqkv, wo, past[b], freq, r[offsets[b]:offsets[b + 1]])
                              for b in range(B)])
        check(y, ref, f"{mode}, step {step}")
    if mode == "pages":  # fewer than there are: the same call, finite and near the full one's
        few = awq.attention(dev(x), pw, po, cache, seqs, dev(freq), residual=dev(r), pages=4)
        assert bool(torch.isfinite(few).all())
