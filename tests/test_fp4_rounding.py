"""The 16-bit quantiser's shortcut: a product with a reciprocal that is rounded up, cut off towards zero, decides every
tie as the exact quotient does. Exact rational arithmetic, all significands."""
from fractions import Fraction as F

import numpy as np


def up(x):
    """The least fp32 that is no less than x > 0."""
    f = np.float32(float(x))
    while F(float(f)) < x:
        f = np.nextafter(f, np.float32(np.inf))
    while F(float(np.nextafter(f, np.float32(0)))) >= x:
        f = np.nextafter(f, np.float32(0))
    return F(float(f))


def cut(x):
    """The largest fp32 that is no more than x > 0."""
    f = np.float32(float(x))
    while F(float(f)) > x:
        f = np.nextafter(f, np.float32(0))
    while F(float(np.nextafter(f, np.float32(np.inf)))) <= x:
        f = np.nextafter(f, np.float32(np.inf))
    return F(float(f))


TIES = [F(1, 4), F(3, 4), F(5, 4), F(7, 4), F(5, 2), F(7, 2), F(5)]


def test_codes():
    for m in range(8, 16):
        s = F(m, 8)
        inv = up(1 / s)
        for tie in TIES:
            assert cut(tie * s * inv) == tie
            for x in (tie * s * (1 - F(1, 4096)), tie * s * (1 + F(1, 4096))):  # nearer no 16-bit value comes
                assert (cut(x * inv) < tie) == (x < tie * s) and cut(x * inv) != tie


def test_block_scales():
    sixth = up(F(1, 6))
    assert float(sixth) == 0.16666667163372039794921875
    for k in range(1, 32, 2):  # ties of E4M3: 5 bits, fewer among its subnormals
        tie = F(k, 16)
        assert cut(6 * tie * sixth) == tie
        for x in (6 * tie * (1 - F(1, 4096)), 6 * tie * (1 + F(1, 4096))):
            assert (cut(x * sixth) < tie) == (x < 6 * tie)


def test_distance_of_16_bit_values():
    """A value of up to 11 significant bits and a tie times a scale, of 7, are equal or 2^-12 of them apart."""
    points = sorted({tie * F(m, 8) for tie in TIES for m in range(8, 16)} | {6 * F(k, 16) for k in range(17, 32, 2)})
    for point in points:
        e = 0
        while point / F(2) ** e >= 2:
            e += 1
        while point / F(2) ** e < 1:
            e -= 1
        step = F(2) ** (e - 10)
        below, above = point // step * step, point // step * step + step
        assert below == point or point - below >= point / 4096
        assert above - point >= point / 4096
        if below == point:
            assert step / 2 >= point / 4096  # the next one down may be of the finer binade
