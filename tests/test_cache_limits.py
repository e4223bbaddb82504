"""Shapes at the limits of a launch are refused on the host: every launch has less than 2^32 threads (no GPU needed: the calls
fail validation, so no pointer is dereferenced)."""
from __future__ import annotations

import pytest

from tests.test_cache_abi import attending, attending_pages, awq, lib  # noqa: F401  (lib: the library's fixture)

# as many sequences, tokens and heads as there may be, over tables so wide that row tiles take the own keys: a workgroup of
# 256 threads for every token and head, and more for the shared keys
MANY = dict(T=65535, B=65536, Hq=256, Hkv=256, D=64, ldq=256 * 64, ldy=256 * 64, width=64, size=32, wsb=1 << 60)


def workspace(lib, shared, **kw):  # noqa: F811
    a = dict(MANY, **kw)
    return lib.awq_attend_workspace_bytes(a["T"], a["B"], a["Hq"], a["Hkv"], a["D"], a["width"], a["size"], shared)


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("shared", [32, 64, 1024])
def test_row_tiles_past_a_launch(lib, shared, D):  # noqa: F811
    assert attending(lib, **dict(MANY, D=D, ldq=256 * D, ldy=256 * D), shared=shared) == awq.AWQ_ERR_SHAPE
    assert workspace(lib, shared, D=D) == 0


def test_what_fits_is_taken(lib):  # noqa: F811
    """(By the workspace's size: parts of both kinds of keys.)"""
    for kw in (dict(B=60000, T=65535 - 5536), dict(width=16), dict(Hq=128, Hkv=128), dict(T=32768, B=32768)):
        assert workspace(lib, 64, **kw) >= 2 * dict(MANY, **kw)["T"] * dict(MANY, **kw)["Hq"] * (64 * 4 + 8), kw


@pytest.mark.parametrize("call", [attending, attending_pages])
def test_scales_past_the_powers_of_two_are_refused(lib, call):  # noqa: F811
    """Times log2(e) they are infinite: every row would be NaN.  (What is taken is told by the check that follows.)"""
    for scale in (2.36e38, 3.4e38):
        assert call(lib, scale=scale) == awq.AWQ_ERR_OPTION, scale
    for scale in (2.35e38, 1e-30, 1e-45):
        assert call(lib, scale=scale, y=0) == awq.AWQ_ERR_NULL, scale
