"""Checks of attention over many keys that a single block of 32 keys left out does not pass.

Element by element, the worst case of fp32 sums over n keys (n * 2^-24 each) is more than what 32 keys of tens of thousands give.
Three checks that do not grow with n:

* the 2-norm.  Weights and results are rounded to fp16, each by 2^-11 of its value at most; the values are independent of
  the weights' roundings, so that the error is 2^-11 of the result's 2-norm for each of the two at most, 2^-11 sqrt 2 = 6.9e-4
  for both, and 2^-10 leaves a factor of 1.4 for what a finite number of channels strays (1024 of them: 3 %) and for
  scores (D * 2^-24 of a few units).  32 keys of n are sqrt(32 / n) of it: 0.022 at 65537.
* queries of 0 and whole values, one channel per block: all weights are equal and a power of two, all sums are whole numbers
  below 2^24, so that only the division (2^-22) and the result's rounding (2^-11) are not exact.
* one block whose keys have all the weight, each block in turn: the mean of its values, by their roundings to fp32
  sums (32 * 2^-24) and the result's rounding.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32


def check_norm(got, ref, what):
    off = np.linalg.norm(got.astype(np.float64) - ref) / np.linalg.norm(ref)
    assert off <= 2.0 ** -10, f"{what}: 2-norm error {off:.2e}"


def whole_values(n, D):
    """[n, D]: block b of 32 keys has 1 to 7 in channel b % D."""
    v = np.zeros((n, D), np.float16)
    block = np.arange(n) // BLOCK
    v[np.arange(n), block % D] = 1 + block // D % 7
    return v


def check_whole(got, v, what):
    """Of equal weights; v [n, D] whole."""
    ref = v.astype(np.float64).sum(0) / len(v)
    assert len(v) * float(v.max()) < 1 << 24
    off = np.abs(got.astype(np.float64) - ref)
    assert np.all(off <= ref * (2.0 ** -11 + 2.0 ** -21) + (ref > 0) * 2.0 ** -25), f"{what}: {np.max(off / np.maximum(ref, 1e-9)):.2e}"


BITS = 12  # of a block's number


def codes(blocks, D):
    """[len(blocks), D]: the bits of each block's number as 1 and -1: the product of two is 12, of different ones 10 at most."""
    out = np.zeros((len(blocks), D), np.float16)
    out[:, :BITS] = 1 - 2 * (np.asarray(blocks)[:, None] >> np.arange(BITS) & 1)
    return out


CODE_SCALE = 16.0  # exp(-2 * 16) of all other blocks' keys: 1e-14 each


def check_block(got, v, block, what):
    """The mean of a block's values."""
    part = v[BLOCK * block:BLOCK * (block + 1)].astype(np.float64)
    ref = part.mean(0)
    tol = np.abs(ref) * 2.0 ** -11 + np.abs(part).mean(0) * 40 * 2.0 ** -24 + len(v) * 1.3e-14 * 6 + 2.0 ** -25
    off = np.abs(got.astype(np.float64) - ref)
    assert np.all(off <= tol), f"{what}, block {block}: {np.max(off / tol):.2f} times the bound"
