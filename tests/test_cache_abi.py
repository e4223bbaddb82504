"""The operators on a paged cache refuse what they cannot take, on the host and before any launch (no GPU needed: every
call below fails validation, so no pointer is dereferenced); and the oracle's own forms agree with hand-worked values
and with a second statement of them."""
from __future__ import annotations

import os

import numpy as np
import pytest

from oracle import cache_oracle as C

awq = pytest.importorskip("bit_weight_only_awq_amd")
torch = pytest.importorskip("torch")

P = [0x7F0000000000 + i * 0x10000000 for i in range(14)]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(awq.LIB_PATH):
        pytest.fail(f"{awq.LIB_PATH} not built; run python -m bit_weight_only_awq_amd.build")
    return awq.load_library()


BATCH = dict(ldq=1024, off=P[1], len=P[2], tab=P[3], width=8, T=4, B=3, Hq=8, Hkv=2, D=128)
PAGES = dict(k=P[4], v=P[5], pages=10, size=16)
OUT = dict(y=P[6], ldy=1024, ws=P[7], wsb=1 << 40)


def ordered(a, names):
    pointers = ("q", "x", "off", "len", "tab", "k", "v", "y", "ws", "freq", "pos", "axis", "bounds", "chosen")
    return [a[n] or None if n in pointers else a[n] for n in names.split()]


def appending(lib, **kw):
    a = dict(BATCH, **PAGES, x=P[0], ldx=1536, freq=P[8], rot=128, inter=0, pos=P[9], axes=3, axis=P[10], y=P[6],
             bounds=P[11], ldq=1024)
    a.update(kw)
    return lib.awq_append_kv(*ordered(a, "x ldx off len tab width T B Hq Hkv D freq rot inter pos axes axis y ldq k v "
                                         "bounds pages size"), None)


def attending(lib, **kw):
    a = dict(BATCH, **PAGES, **OUT, q=P[0], scale=0.1, shared=32)
    a.update(kw)
    return lib.awq_attend(*ordered(a, "q ldq off len tab width T B Hq Hkv D scale shared k v pages size y ldy ws wsb"),
                          None)


def selecting(lib, **kw):
    a = dict(BATCH, **PAGES, **OUT, q=P[0], bounds=P[11], count=4, first=1, recent=1, chosen=P[12])
    a.update(kw)
    return lib.awq_select_pages(*ordered(a, "q ldq off len tab width T B Hq Hkv D bounds pages size count first recent "
                                            "chosen ws wsb"), None)


def attending_pages(lib, **kw):
    a = dict(BATCH, **PAGES, **OUT, q=P[0], scale=0.1, count=4, chosen=P[12])
    a.update(kw)
    return lib.awq_attend_pages(*ordered(a, "q ldq off len tab width T B Hq Hkv D scale chosen count k v pages size y "
                                            "ldy ws wsb"), None)


CALLS = [appending, attending, selecting, attending_pages]


@pytest.mark.parametrize("call", CALLS)
def test_what_all_refuse(lib, call):
    for kw in (dict(T=0), dict(T=-3), dict(B=0), dict(B=(1 << 16) + 1), dict(Hkv=0), dict(Hkv=3), dict(Hq=0),
               dict(Hq=1026), dict(T=1 << 22), dict(width=0), dict(width=1 << 27), dict(pages=0), dict(size=8),
               dict(size=48), dict(size=512), dict(size=0), dict(ldq=1016), dict(ldq=1028), dict(ldq=(1 << 21) + 8),
               dict(ldq=-1024)):
        assert call(lib, **kw) == awq.AWQ_ERR_SHAPE, kw
    for D in (0, 32, 80, 127, 160, 512):
        assert call(lib, D=D) == awq.AWQ_ERR_UNSUPPORTED, D
    for name in ("off", "len", "tab"):
        assert call(lib, **{name: 0}) == awq.AWQ_ERR_NULL, name
        assert call(lib, **{name: BATCH[name] + 2}) == awq.AWQ_ERR_ALIGN, name


def test_append_refusals(lib):
    for kw in (dict(ldx=1528), dict(ldx=1540)):
        assert appending(lib, **kw) == awq.AWQ_ERR_SHAPE, kw
    for kw in (dict(rot=-16), dict(rot=8), dict(rot=72), dict(rot=144), dict(axes=0), dict(axes=17)):
        assert appending(lib, **kw) == awq.AWQ_ERR_OPTION, kw
    for name in ("x", "y", "k", "v", "freq", "axis"):
        assert appending(lib, **{name: 0}) == awq.AWQ_ERR_NULL, name
    for name, at in (("x", P[0]), ("y", P[6]), ("k", P[4]), ("v", P[5]), ("bounds", P[11])):
        assert appending(lib, **{name: at + 8}) == awq.AWQ_ERR_ALIGN, name
    for name, at in (("freq", P[8]), ("pos", P[9]), ("axis", P[10])):
        assert appending(lib, **{name: at + 2}) == awq.AWQ_ERR_ALIGN, name


@pytest.mark.parametrize("call", [attending, attending_pages])
def test_attend_refusals(lib, call):
    for kw in (dict(ldy=1016), dict(ldy=1030)):
        assert call(lib, **kw) == awq.AWQ_ERR_SHAPE, kw
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(lib, scale=scale) == awq.AWQ_ERR_OPTION, scale
    for name in ("q", "k", "v", "y"):
        assert call(lib, **{name: 0}) == awq.AWQ_ERR_NULL, name
        assert call(lib, **{name: dict(q=P[0], k=P[4], v=P[5], y=P[6])[name] + 8}) == awq.AWQ_ERR_ALIGN, name


def test_attend_shared_and_workspace(lib):
    for shared in (-16, 8, 17, 144):
        assert attending(lib, shared=shared) == awq.AWQ_ERR_OPTION, shared
    need = lib.awq_attend_workspace_bytes(4, 3, 8, 2, 128, 8, 16, 32)
    if need:
        assert attending(lib, wsb=need - 1) == awq.AWQ_ERR_WORKSPACE
        assert attending(lib, ws=0) == awq.AWQ_ERR_NULL and attending(lib, ws=P[7] + 8) == awq.AWQ_ERR_ALIGN
    for bad in ((0, 3, 8, 2, 128, 8, 16, 32), (4, 0, 8, 2, 128, 8, 16, 0), (4, 3, 8, 3, 128, 8, 16, 0),
                (4, 3, 8, 2, 80, 8, 16, 0), (4, 3, 8, 2, 128, 0, 16, 0), (4, 3, 8, 2, 128, 8, 24, 0),
                (4, 3, 8, 2, 128, 8, 16, -16)):
        assert lib.awq_attend_workspace_bytes(*bad) == 0, bad


def test_pages_refusals(lib):
    for kw in (dict(count=0), dict(count=-1), dict(first=-1), dict(recent=0), dict(first=3, recent=2),
               dict(first=2147483647, recent=2147483647), dict(count=1 << 29)):
        assert selecting(lib, **kw) == awq.AWQ_ERR_OPTION, kw
    for name in ("q", "bounds", "chosen"):
        assert selecting(lib, **{name: 0}) == awq.AWQ_ERR_NULL, name
    for name, at in (("q", P[0] + 8), ("bounds", P[11] + 8), ("chosen", P[12] + 2)):
        assert selecting(lib, **{name: at}) == awq.AWQ_ERR_ALIGN, name
    need = lib.awq_select_pages_workspace_bytes(4, 2, 5000, 4)
    assert need > 0 and lib.awq_select_pages_workspace_bytes(4, 2, 8, 8) == 0
    assert lib.awq_select_pages_workspace_bytes(4, 2, 512, 4) == 0 and lib.awq_select_pages_workspace_bytes(4, 2, 513, 4) > 0
    assert selecting(lib, width=5000, wsb=need - 1) == awq.AWQ_ERR_WORKSPACE
    assert selecting(lib, width=5000, ws=0, wsb=need) == awq.AWQ_ERR_NULL
    for bad in ((0, 2, 8, 4), (4, 0, 8, 4), (4, 2, 0, 4), (4, 2, 8, 0), (1 << 24, 2, 8, 4)):
        assert lib.awq_select_pages_workspace_bytes(*bad) == 0, bad
    for kw in (dict(count=0), dict(count=1 << 29)):
        assert attending_pages(lib, **kw) == awq.AWQ_ERR_OPTION, kw
    assert attending_pages(lib, chosen=0) == awq.AWQ_ERR_NULL
    assert attending_pages(lib, chosen=P[12] + 2) == awq.AWQ_ERR_ALIGN
    need = lib.awq_attend_pages_workspace_bytes(4, 8, 2, 128, 16, 4)
    if need:
        assert attending_pages(lib, wsb=need - 1) == awq.AWQ_ERR_WORKSPACE and attending_pages(lib, ws=0) == awq.AWQ_ERR_NULL
    for bad in ((0, 8, 2, 128, 16, 4), (4, 8, 3, 128, 16, 4), (4, 8, 2, 80, 16, 4), (4, 8, 2, 128, 8, 4),
                (4, 8, 2, 128, 16, 0)):
        assert lib.awq_attend_pages_workspace_bytes(*bad) == 0, bad


def test_binding_refusals():
    half = lambda *shape: torch.zeros(shape, dtype=torch.float16)  # noqa: E731
    cache = awq.KvCache(half(10, 2, 16, 128), half(10, 2, 16, 128), None)
    seqs = awq.Sequences(torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                         torch.zeros((2, 4), dtype=torch.int32))
    q = half(4, 1024)
    for bad in (q, q.float(), q[:, :1000], q[:, :0], half(4, 384), half(4, 8, 128)):  # on the host, type, widths
        with pytest.raises(ValueError):
            awq.attend(bad, cache, seqs)
    with pytest.raises(ValueError):
        awq.append_kv(half(4, 512), cache, seqs)  # no room for queries
    with pytest.raises(ValueError, match="keys and values"):
        awq.attend(q, cache._replace(v=half(10, 2, 16, 64)), seqs)
    with pytest.raises(ValueError):
        awq.attend_pages(q, cache, seqs, torch.zeros((4, 3, 5), dtype=torch.int32))


def test_attention_refuses_chosen_pages_of_a_shared_prefix():
    with pytest.raises(ValueError, match="shared must be 0"):
        awq.attention(torch.zeros((1, 64), dtype=torch.float16), None, None, None, None, shared=16, pages=4)


def test_oracle_by_hand():
    q = np.array([1.0, -2.0])
    k, v = np.array([[0.0, 0.0], [np.log(3.0), 0.0]]), np.array([[4.0, 0.0], [0.0, 8.0]])
    y, _ = C.attend_row(q, k, v, 1.0)
    assert np.allclose(y, [1.0, 6.0])
    assert np.all(C.attend_row(q, k[:0], v[:0], 1.0)[0] == 0)
    bounds = np.array([[[-1.0, -3.0], [2.0, 5.0]], [[0.0, 0.0], [9.0, 0.0]]])
    assert np.allclose(C.scores(q[None], bounds), [2 + 6, 9])
    # the largest score that a key within the bounds has, by trying the corners
    corners = [np.dot(q, [a, b]) for a in (-1, 2) for b in (-3, 5)]
    assert C.scores(q[None], bounds)[0] == max(corners)
    assert C.select(q[None], np.repeat(bounds, [2, 2], 0), 4, 2, 0, 1).tolist() == [2, 3]
    assert C.select(q[None], bounds, 2, 3, 1, 1).tolist() == [0, 1, -1]
    x = np.array([[[1.0, 0.0, 2.0, 5.0]]])
    turned, _ = C.rotate(x, np.array([1]), np.array([np.pi / 2]), False)
    assert np.allclose(turned, [[[0.0, 1.0, 2.0, 5.0]]])
    turned, _ = C.rotate(x, np.array([2]), np.array([np.pi / 2, 0.0]), False)
    assert np.allclose(turned, [[[-1.0, 0.0, -2.0, 5.0]]])
    turned, _ = C.rotate(x, np.array([1]), np.array([0.0, np.pi / 2]), True)
    assert np.allclose(turned, [[[1.0, 0.0, -5.0, 2.0]]])
    seq, place = C.places([0, 2, 2, 3], [5, 0, 1], 4)
    assert seq.tolist() == [0, 0, 2, -1] and place.tolist() == [3, 4, 0, -1]
