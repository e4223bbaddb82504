"""A decoder block's attention to chosen pages, step after step, against fp64 of the same block: pages chosen from bounds of
the keys as they are stored, with numbers of first and recent pages other than the defaults."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import cache_oracle as C
from tests import _gpu as G
from tests._fused import halves, packed_layer

torch = pytest.importorskip("torch")

K, HQ, HKV, D, S = 512, 8, 2, 64, 16
PAGES, FIRST, RECENT = 5, 1, 2
SEED = 0
FREQ = (10000.0 ** (-np.arange(0, D, 2) / D)).astype(np.float32)
STEPS = ([90, 150, 40], [1, 1, 1], [1, 1, 1], [2, 1, 3], [1, 1, 1], [17, 1, 2], [1, 1, 1])


def rotated_rows(x, wqkv, at):
    n = len(x)
    rows = (x.astype(np.float64) @ wqkv.T).astype(np.float16).astype(np.float64).reshape(n, HQ + 2 * HKV, D)
    angle = (at + np.arange(n))[:, None] * FREQ.astype(np.float64)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    a, b = rows[:, :HQ + HKV, :D // 2].copy(), rows[:, :HQ + HKV, D // 2:].copy()
    rows[:, :HQ + HKV] = np.concatenate([a * c - b * s, b * c + a * s], 2)
    return rows.astype(np.float16)


def choice(q, k, place):
    """Pages of queries q [G, D] at `place`, of one key head's keys k [n, D]; and by how much the scores decide, as a
    multiple of what roundings of queries and bounds, an ulp each (2^-10), move them in the mean square."""
    have = place // S + 1
    bounds = np.stack([np.stack([k[S * p:S * p + S].min(0), k[S * p:S * p + S].max(0)]) for p in range(have)])
    chosen = C.select(q, bounds, have, PAGES, FIRST, RECENT)
    clear = np.inf
    if have > PAGES:
        middle = bounds[FIRST:have - RECENT]
        score = np.sort(C.scores(q, middle))[::-1]
        wide = np.abs(middle.astype(np.float64)).max(1)
        moved = 2.0 ** -10 * np.sqrt(2 * ((np.abs(q.astype(np.float64))[:, None] * wide) ** 2).sum((0, 2)).max())
        n = PAGES - FIRST - RECENT
        clear = (score[n - 1] - score[n]) / moved
    return chosen, clear


def reference(x, wqkv, wo, past, residual):
    n, at = len(x), len(past[0])
    rows = rotated_rows(x, wqkv, at)
    k = past[0] = np.concatenate([past[0], rows[:, HQ:HQ + HKV]])
    v = past[1] = np.concatenate([past[1], rows[:, HQ + HKV:]])
    y, clear, few = np.zeros((n, HQ, D)), np.inf, 0
    for i in range(n):
        for h in range(HKV):
            group = range(h * HQ // HKV, (h + 1) * HQ // HKV)
            chosen, c = choice(rows[i, group], k[:, h], at + i)
            clear, few = min(clear, c), few + (c < np.inf)
            keys = np.array([j for p in chosen if p >= 0 for j in range(S * p, min(S * p + S, at + i + 1))])
            for g in group:
                y[i, g] = C.attend_row(rows[i, g], k[keys, h], v[keys, h], D ** -0.5)[0]
    return y.reshape(n, -1) @ wo.T + residual.astype(np.float64), clear, few


def steps(wqkv, wo, seed):
    """(new tokens, x, residual, lengths, expected) of each step."""
    B = len(STEPS[0])
    past = [[np.zeros((0, HKV, D), np.float16)] * 2 for _ in range(B)]
    lengths = np.zeros(B, int)
    for step, new in enumerate(STEPS):
        x, r = halves((sum(new), K), 100 * seed + step), halves((sum(new), K), 100 * seed + 50 + step)
        at = np.concatenate([[0], np.cumsum(new)])
        lengths = lengths + new
        out = [reference(x[at[b]:at[b + 1]], wqkv, wo, past[b], r[at[b]:at[b + 1]]) for b in range(B)]
        yield (new, x, r, lengths.copy(), np.concatenate([o[0] for o in out]), min(o[1] for o in out), sum(o[2] for o in out))


@pytest.mark.gpu
def test_block_over_steps_with_chosen_pages():
    awq = G.lib()
    pw, wqkv = packed_layer(awq, (HQ + 2 * HKV) * D, K, 128, True, 3)
    po, wo = packed_layer(awq, K, HQ * D, 64, False, 4)
    B = len(STEPS[0])
    cache = awq.kv_cache(60, HKV, D, S, bounds=True)
    for t in cache:
        t.fill_(float("nan"))
    tables = np.random.default_rng(5).permutation(60)[:B * 16].reshape(B, 16)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).cuda()  # noqa: E731
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    for step, (new, x, r, lengths, ref, clear, _) in enumerate(steps(wqkv, wo, SEED)):
        assert clear > 1.0, "inputs whose choice the roundings may turn"
        seqs = awq.Sequences(i32(np.concatenate([[0], np.cumsum(new)])), i32(lengths), i32(tables))
        y = awq.attention(dev(x), pw, po, cache, seqs, dev(FREQ), residual=dev(r), pages=PAGES, first=FIRST, recent=RECENT)
        y = y.cpu().numpy().astype(np.float64)
        # (five roundings to fp16 on the way, 2^-11 / sqrt 3 each in the mean square, and scores of a few units that turn
        # 2^-11 of themselves into as much of a weight: 1e-3; twice that is allowed)
        assert np.linalg.norm(y - ref) <= 2e-3 * np.linalg.norm(ref), f"step {step}"
        # and no single row far off (with other pages a row is off by 7 % of itself at least, tried with other `first` and `recent`)
        worst = np.max(np.linalg.norm(y - ref, axis=1) / np.linalg.norm(ref, axis=1))
        assert worst <= 6e-3, f"step {step}: a row is off by {worst:.1e}"
