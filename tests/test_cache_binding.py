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
