"""The MXFP4 oracle in whole numbers, and the arithmetic behind what the header promises of codes."""
from fractions import Fraction
from math import isqrt, sqrt

import numpy as np
import pytest

from oracle import mx


@pytest.mark.parametrize("block", [128, 256, 512])
@pytest.mark.parametrize("unit", [0, -9, -140, 110])
def test_whole_numbers_agree_with_float64(block, unit):
    # sums of few bits, which float64 decides like the exact ones
    rng = np.random.default_rng(block)
    x = np.rint(40 * rng.standard_normal((3, 1024))).astype(np.int64)
    x[2, :512] = 0
    codes, scales = mx.quantize_whole(x, block, unit)
    want, want_s = mx.quantize(mx.rotate(np.ldexp(x.astype(float), unit), block))
    assert np.array_equal(scales, want_s) and np.array_equal(codes, want)


def test_a_tie_and_its_neighbours():
    x = np.zeros((1, 256), np.int64)
    x[0, :2] = 20 << 30, 1  # 1.25, 5 of the scale's quarters... and 2^-34 more or less
    codes, scales = mx.quantize_whole(x, 256, -30)
    assert set(codes[0]) == {7, 6} and (scales == 125).all()
    assert (codes[0, ::2] == 7).all() and (codes[0, 1::2] == 6).all()


@pytest.mark.parametrize("bits,holds", [(46, True), (48, False)])
def test_whole_sums_keep_their_distance_from_borders(bits, holds):
    # u / sqrt(128) and u / sqrt(512) against m 2^k: u against m 2^k sqrt(2).  The roundings of 1 / sqrt(block) and of the
    # product are 2^-53 each, relative to the value.
    P = 200
    nearest = 1.0
    for m in (1, 3, 5, 7):
        for k in range(-4, bits):
            border = isqrt(2 * m * m << 2 * P) << k if k >= 0 else isqrt(2 * m * m << 2 * P) >> -k
            for u in ((border >> P), (border >> P) + 1):
                if 0 < u < 2 ** bits:
                    nearest = min(nearest, float(Fraction(abs((u << P) - border), border)))
    assert (nearest > 2.0 ** -52) == holds
    for block in (128, 512):
        assert abs(Fraction(1 / sqrt(block)) ** 2 * block - 1) < Fraction(1, 2 ** 52)
