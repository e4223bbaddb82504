"""The binding of the operators on a paged cache: what it refuses, as which error, and before anything is written (no GPU
needed)."""
from __future__ import annotations

import pytest

awq = pytest.importorskip("bit_weight_only_awq_amd")
torch = pytest.importorskip("torch")

half = lambda *shape: torch.zeros(shape, dtype=torch.float16)  # noqa: E731
whole = lambda *shape: torch.zeros(shape, dtype=torch.int32)  # noqa: E731


def cache(pages=10, heads=2, size=16, dim=128, bounds=True):
    return awq.KvCache(half(pages, heads, size, dim), half(pages, heads, size, dim),
                       half(pages, heads, 2, dim) if bounds else None)


def sequences(B=2, width=4):
    return awq.Sequences(whole(B + 1), whole(B), whole(B, width))


@pytest.fixture
def calls(monkeypatch):
    """The calls of `attention` that write, by name; layers give zeros."""
    made = []

    def layer(x, pw, bias=None, **kw):
        made.append("layer")
        return half(x.shape[0], pw.N)

    monkeypatch.setattr(awq, "linear_fused", layer)
    monkeypatch.setattr(awq, "append_kv", lambda qkv, cache, *a, **kw: made.append("append") or half(qkv.shape[0], 1024))
    for name in ("attend", "attend_pages", "select_pages"):
        monkeypatch.setattr(awq, name, lambda q, *a, **kw: made.append("attend") or q)
    return made


def weight(N, K):
    return awq.PackedWeight(None, None, None, N, K, 128, True)


QKV, O = weight(1536, 512), weight(512, 1024)


def block(**kw):
    a = dict(x=half(3, 512), qkv=QKV, o=O, cache=cache(), seqs=sequences())
    a.update(kw)
    return awq.attention(**a)


def test_attention_runs_its_calls(calls):
    for kw in ({}, dict(shared=32), dict(pages=3), dict(pages=4, first=0, recent=4),
               dict(scale=0.5), dict(cache=cache(bounds=False)), dict(shared=64)):
        calls.clear()
        block(**kw)
        assert calls[:2] == ["layer", "append"] and calls[-1] == "layer", kw


@pytest.mark.parametrize("kw", [
    dict(pages=4, cache=cache(bounds=False)),                                        # nothing to choose from
    dict(pages=4, cache=cache()._replace(bounds=half(10, 2, 2, 64))),                # bounds of another cache
    dict(pages=1), dict(pages=2, first=2), dict(pages=4, recent=0), dict(pages=4, first=-1), dict(pages=-3),
    dict(pages=1 << 32), dict(pages=4, first=1 << 32), dict(pages=4, recent=1 << 32),
    dict(pages=1 << 28), dict(pages=(1 << 30) // 16 + 1),                            # keys past 2^30
    dict(shared=8), dict(shared=-16), dict(shared=80), dict(shared=1 << 32), dict(shared=16, pages=4),
    dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=1e-50),
    dict(scale=1e39), dict(scale=2.4e38), dict(pages=4, scale=0.0),
    dict(residual=half(2, 512)), dict(residual=half(3, 520)), dict(residual=torch.zeros((3, 512))),
    dict(residual=half(3, 1024)[:, ::2]),
    dict(o=weight(512, 768)), dict(qkv=weight(1024, 512)), dict(qkv=weight(512, 512)), dict(qkv=weight(1500, 512)),
])
def test_attention_refuses_before_it_writes(calls, kw):
    with pytest.raises((ValueError, awq.AwqError)):
        block(**kw)
    assert "append" not in calls


def test_many_rows_are_refused_before_they_are_written(calls):
    for kw, T, N, K in ((dict(pages=4, cache=cache(dim=64)), 1 << 21, 6 * 64, 128),       # 2^22 choices
                        (dict(pages=2048, cache=cache(dim=64)), 1 << 19, 6 * 64, 128),    # 2^31 chosen pages
                        (dict(pages=1024, cache=cache(dim=64, size=64)), 1 << 18, 6 * 64, 128),  # 2^30 units of work
                        (dict(shared=16, cache=cache(heads=256, dim=64), seqs=sequences(65536, 128)), 65535, 768 * 64, 16384)):
        with pytest.raises(awq.AwqError):
            block(x=half(1, 8).expand(T, 8), qkv=weight(N, 8), o=weight(8, K), **kw)
        assert "layer" not in calls


@pytest.mark.parametrize("call", [
    lambda n: awq.attend(half(4, 1024), cache(), sequences(), shared=n),
    lambda n: awq.select_pages(half(4, 1024), cache(), sequences(), n),
    lambda n: awq.select_pages(half(4, 1024), cache(), sequences(), 4, first=n),
    lambda n: awq.select_pages(half(4, 1024), cache(), sequences(), 4, recent=n)])
@pytest.mark.parametrize("n", [1 << 31, 1 << 32, (1 << 32) + 1, -(1 << 32) + 1, -(1 << 31) - 1])
def test_numbers_past_32_bits_are_refused(call, n):
    """(They would arrive as their lowest 32 bits.)"""
    with pytest.raises(awq.AwqError) as e:
        call(n)
    assert e.value.status == awq.AWQ_ERR_OPTION


@pytest.mark.parametrize("bad", [cache(heads=0), cache(dim=0), cache(size=0), cache()._replace(k=half(2, 16, 128)),
                                 cache()._replace(v=half(10, 2, 16, 64)), cache(pages=0)])
def test_caches_of_no_size_are_value_errors(bad):
    for call in (lambda: awq.attend(half(4, 1024), bad, sequences()), lambda: awq.append_kv(half(4, 1536), bad, sequences()),
                 lambda: awq.select_pages(half(4, 1024), bad, sequences(), 4),
                 lambda: awq.attend_pages(half(4, 1024), bad, sequences(), whole(4, 2, 3)),
                 lambda: awq.attention(half(3, 512), QKV, O, bad, sequences())):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("bad", [sequences()._replace(lengths=torch.zeros((), dtype=torch.int32)),
                                 sequences()._replace(lengths=whole(2, 1)), sequences()._replace(tables=whole(8)),
                                 sequences()._replace(offsets=torch.zeros((), dtype=torch.int32)),
                                 sequences()._replace(offsets=whole(2))])
def test_sequences_of_other_shapes_are_value_errors(bad, monkeypatch):
    monkeypatch.setattr(awq, "_rows2d", lambda t, rows, width, what: (0, width))  # (the rows are taken to be on the GPU)
    for call in (lambda: awq.attend(half(4, 1024), cache(), bad), lambda: awq.append_kv(half(4, 1536), cache(), bad),
                 lambda: awq.select_pages(half(4, 1024), cache(), bad, 4),
                 lambda: awq.attend_pages(half(4, 1024), cache(), bad, whole(4, 2, 3))):
        with pytest.raises(ValueError, match="seqs"):
            call()


def test_pages_of_another_shape_are_value_errors():
    for bad in (whole(4, 2), whole(4, 3, 5), whole(3, 2, 5), whole(4), torch.zeros((), dtype=torch.int32)):
        with pytest.raises(ValueError):
            awq.attend_pages(half(4, 1024), cache(), sequences(), bad)
    with pytest.raises(ValueError):
        awq.attend_pages(torch.zeros((), dtype=torch.float16), cache(), sequences(), whole(4, 2, 3))


def test_a_cache_without_pages_is_one_where_there_are_no_tokens(monkeypatch):
    monkeypatch.setattr(awq, "_rows2d", lambda t, rows, width, what: (0, width))  # (the rows are taken to be on the GPU)
    monkeypatch.setattr(awq, "_handle", lambda t: 0)
    assert awq.attend(half(0, 1024), cache(pages=0), sequences()).shape == (0, 1024)
    assert awq.append_kv(half(0, 1536), cache(pages=0), sequences()).shape == (0, 1024)
    assert awq.select_pages(half(0, 1024), cache(pages=0), sequences(), 4).shape == (0, 2, 4)
