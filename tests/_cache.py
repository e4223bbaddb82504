"""Inputs and checks shared by the tests of the operators on a paged cache."""
from __future__ import annotations

import numpy as np

from oracle import cache_oracle as C
from tests import _gpu as G


class Batch:
    """Sequences on a paged cache, on the host: unused slots and pages hold NaN and infinities, table entries past a
    sequence's pages hold anything, `pad` rows follow the last sequence."""

    def __init__(self, new, past, Hq, Hkv, D, S, shared=0, pad=0, seed=0, scale=1.0, width=None):
        rng = self.rng = np.random.default_rng([23, seed, D, S])
        self.new, self.Hq, self.Hkv, self.D, self.S, self.shared = list(new), Hq, Hkv, D, S, shared
        self.lengths = [shared + p + n for n, p in zip(new, past)]
        self.B, self.T = len(new), sum(new) + pad
        own = [-(-n // S) - shared // S for n in self.lengths]
        common = shared // S
        pool = common + sum(max(0, n) for n in own) + 2
        order = rng.permutation(pool)
        self.width = width or common + max(max(own), 0) + 1
        self.tables = rng.choice([-7, 1 << 30, -(1 << 31), 3], (self.B, self.width)).astype(np.int64)
        self.tables[:, :common] = order[:common]
        at = common
        for b, n in enumerate(own):
            n = max(n, 0)
            self.tables[b, common:common + n] = order[at:at + n]
            at += n
        self.offsets = np.concatenate([[0], np.cumsum(self.new)])
        self.seq, self.place = C.places(self.offsets, self.lengths, self.T)
        self.k = (rng.standard_normal((pool, Hkv, S, D)) * scale).astype(np.float16)
        self.v = rng.standard_normal((pool, Hkv, S, D)).astype(np.float16)
        used = np.zeros((pool, S), bool)
        for b, n in enumerate(self.lengths):
            for i in range(-(-n // S)):
                used[self.tables[b, i], :min(S, n - i * S)] = True
        junk = np.array([np.nan, np.inf, -np.inf, 65504], np.float16)
        for a in (self.k, self.v):
            a.transpose(0, 2, 1, 3)[~used] = rng.choice(junk, ((~used).sum(), Hkv, D))
        self.used = used
        self.q = (rng.standard_normal((self.T, Hq * D)) * scale).astype(np.float16)
        self.q[sum(new):] = np.nan

    def keys(self, b, h, n, which="k"):
        """The first n keys (values) of sequence b, key head h."""
        a, S = getattr(self, which), self.S
        pages = self.tables[b, :-(-n // S)] if n else []
        return np.concatenate([a[p, h] for p in pages])[:n] if n else np.zeros((0, self.D), np.float16)

    def device(self):
        import torch

        awq = G.lib()
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(np.asarray(a).astype(np.int32))).cuda()  # noqa: E731
        return (awq.KvCache(G.dev_f16(self.k), G.dev_f16(self.v), None),
                awq.Sequences(i32(self.offsets), i32(self.lengths), i32(self.tables)))

    def expected(self, scale=None, chosen=None, rows=None):
        """(y, bound, rows) of `rows` (a few, spread, if None)."""
        scale = self.D ** -0.5 if scale is None else scale
        real = [t for t in range(self.T) if self.seq[t] >= 0]
        if rows is None:
            rows = sorted(set(real[:: max(1, len(real) // 24)] + real[:1] + real[-1:]))
        G_, D = self.Hq // self.Hkv, self.D
        y, e = np.zeros((len(rows), self.Hq * D)), np.zeros((len(rows), self.Hq * D))
        for i, t in enumerate(rows):
            for h in range(self.Hkv):
                n = max(0, int(self.place[t]) + 1)
                k, v = self.keys(self.seq[t], h, n), self.keys(self.seq[t], h, n, "v")
                if chosen is not None:
                    at = [j for p in chosen[t, h] if p >= 0 for j in range(p * self.S, min(n, (p + 1) * self.S))]
                    k, v = k[at], v[at]
                for g in range(h * G_, (h + 1) * G_):
                    part = slice(g * D, (g + 1) * D)
                    y[i, part], e[i, part] = C.attend_row(self.q[t, part], k, v, scale)
        return y, e, rows

    def check(self, y, what, scale=None, chosen=None, rows=None):
        ref, bound, rows = self.expected(scale, chosen, rows)
        got = y.cpu().numpy().astype(np.float64)[rows]
        assert np.all(np.isfinite(got)), f"{what}: non-finite output"
        off = np.abs(got - ref)
        worst = float(np.max(off / np.maximum(bound, 1e-30))) if off.size else 0.0
        assert worst <= 1.0, f"{what}: {worst:.2f} times the bound"
