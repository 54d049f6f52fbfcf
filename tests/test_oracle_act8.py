"""Pins of the oracle's 8-bit checkpoints: exact rounding against rational
arithmetic (ties included), the error bound of a block, and the special
blocks."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import act8


def _bf16(rng, shape, scale=1.0):
    x = (rng.standard_normal(shape) * scale).astype(np.float32)
    return ((x.view(np.uint32) & 0xFFFF0000).view(np.float32)).astype(np.float64)


def _half_even(fr):
    lo = fr.numerator // fr.denominator
    rest = fr - lo
    if rest > Fraction(1, 2) or (rest == Fraction(1, 2) and lo % 2):
        return lo + 1
    return lo


@pytest.mark.parametrize("seed,scale", [(0, 1.0), (1, 2.0 ** -120), (2, 2.0 ** 120)])
def test_codes_are_the_exact_quotients_rounded(seed, scale):
    x = _bf16(np.random.default_rng(seed), (2, 128), scale)
    codes, _ = act8.quantize(x)
    for m in range(2):
        for b in range(2):
            blk = [Fraction(v) for v in x[m, 64 * b:64 * b + 64]]
            a = max(abs(v) for v in blk)
            want = [_half_even(127 * v / a) for v in blk]
            assert list(codes[m, 64 * b:64 * b + 64]) == want


def test_ties_go_to_the_even_code():
    # a = 254: 127 x / a = x / 2, so odd x are ties
    x = np.zeros((1, 64))
    x[0, 0], x[0, 1:9] = 254.0, [1, 3, 5, 7, -1, -3, -5, 2]
    codes, scale = act8.quantize(x)
    assert list(codes[0, :9]) == [127, 0, 2, 2, 4, 0, -2, -2, 1]
    assert scale[0, 0] == np.float32(2.0) and not scale[0, 1:].any()


def test_error_of_a_block_is_half_a_step():
    x = _bf16(np.random.default_rng(3), (40, 192))
    codes, scale = act8.quantize(x)
    a = np.abs(x.reshape(40, 3, 64)).max(2)
    err = np.abs(act8.dequantize(codes, scale) - x).reshape(40, 3, 64).max(2)
    # half a step, and two roundings to float32 of values of at most a
    assert np.all(err <= a / 254 + a * 2.0 ** -23)
    assert np.all(np.abs(codes.reshape(40, 3, 64)).max(2) == 127)


def test_special_blocks():
    x = np.zeros((3, 128))
    x[1, 5], x[2, 70] = np.inf, np.nan
    x[1, 64:] = 1.0
    codes, scale = act8.quantize(x)
    assert not codes[0].any() and not codes[1, :64].any() and not codes[2].any()
    assert np.isnan(scale[0, 1]) and np.isnan(scale[1, 2])
    assert scale[0, 0] == 0 and scale[0, 2] == 0 and scale[1, 1] == np.float32(1) / np.float32(127)
    assert scale.shape == (2, 32) and not scale[:, 3:].any()
