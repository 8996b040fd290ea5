"""Frequencies as 64-bit fractions of a turn: the nearest to the double's exact quotient by 2 pi."""
from fractions import Fraction

import numpy as np
import pytest

import bit_block_scaled_gb300 as moe
from bit_block_scaled_gb300 import build as B
from oracle import rope as R

PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798214808651")
TWO_PI = 2 * PI


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return moe.load()


def off(f, turns):
    """How far turns is from f / (2 pi) 2^64, modulo 2^64."""
    d = (Fraction(float(f)) / TWO_PI * 2 ** 64 - int(turns)) % 2 ** 64
    return float(min(d, 2 ** 64 - d))


def frequencies():
    rng = np.random.default_rng(0)
    f = [1.0, 0.1, 1 / 3, 1e-4, 7.5, 1e6, 2.0 ** 30, 1e-18, 5e-324, 0.0, np.pi, 2 * np.pi, np.nextafter(2 * np.pi, 0), 1e-17]
    f += list(rng.random(200)) + list(10.0 ** rng.uniform(-12, 8, 200))
    for base in (10000.0, 500000.0):
        f += list(R.frequencies(128, base=base)[0])
    return np.array(f)


def test_to_the_nearest():
    """Half a step, and the second double's 2^-106 of up to 2^30 turns' worth of steps."""
    f = frequencies()
    for x in (f, -f):
        turns = moe.moe_rope_turns(x)
        assert max(off(a, b) for a, b in zip(x, turns)) <= 0.5 + 2.0 ** -11


def test_negative_ones_turn_back():
    f = frequencies()
    with np.errstate(over="ignore"):
        assert (moe.moe_rope_turns(f) + moe.moe_rope_turns(-f) == 0).all()


def test_huge_ones_are_taken():
    """Doubles of 2^54 and more are whole multiples of 4: what is left of the turn is what two doubles give."""
    for f in (2.0 ** 60, 1e300, -1e300, float(np.finfo(np.float64).max)):
        assert moe.moe_rope_turns([f]).shape == (1,)


@pytest.mark.parametrize("kw", [dict(), dict(base=500000.0), dict(scaling="ntk", factor=8.0),
                                dict(scaling="yarn", factor=32.0, base=150000.0, truncate=False),
                                dict(scaling="llama3", factor=8.0, base=500000.0), dict(scaling="linear", factor=4.0)])
def test_tables(kw):
    """The library's own frequencies are doubles a few last bits apart from the oracle's; the fastest pair's is 1 or 1 over a
    factor that is a power of two, exactly."""
    turns, _ = moe.moe_rope_table(128, **kw)
    f, _ = R.frequencies(128, **kw)
    assert off(f[0], turns[0]) <= 0.5 + 2.0 ** -11
    assert all(off(a, b) <= 0.5 + 2.0 ** -11 + 8 * 2.0 ** 11 * a / 6 for a, b in zip(f, turns))
