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
                 lambda: awq.attend_pages(half(4, 1024), bad, sequences(), whole(4, 2, 3))):
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
