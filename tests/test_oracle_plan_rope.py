"""Pins of oracle/plan.py and oracle/rope.py, and the library's host table of frequencies against the oracle's."""
import math

import numpy as np
import pytest

import bit_block_scaled_gb300 as moe
from bit_block_scaled_gb300 import build as B
from oracle import plan as P
from oracle import rope as R


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return moe.load()


def test_a_worked_plan():
    table = np.array([[0, 1, -1, -1], [2, -1, -1, -1], [3, 4, 5, -1]])
    free = [6, 7, 8, -1, -1, -1, -1, -1, -1]
    p = P.batch_plan([1, 40, -1], [32, 16, 40], table, free, 3, 16, 50)
    # sequence 2 gives back 3, 4, 5 on top of 6, 7, 8; sequence 0 takes 5, sequence 1 takes 4, 3, 8
    assert list(p["free"][:6]) == [6, 7, 8, 3, 4, 5] and p["count"] == 2
    assert list(p["table"][0]) == [0, 1, 5, -1] and list(p["table"][1]) == [2, 4, 3, 8]
    assert list(p["lens"]) == [33, 56, 0] and list(p["offsets"]) == [0, 1, 41, 41] and p["errors"] == 0
    assert p["slots"][0] == 5 * 16 and p["positions"][0] == 32
    assert p["slots"][1] == 4 * 16 and p["slots"][17] == 3 * 16 and p["slots"][40] == 8 * 16 + 7
    assert list(p["seq_ids"][[0, 1, 40, 41]]) == [0, 1, 1, -1] and (p["slots"][41:] == -1).all()


def test_all_or_nothing():
    table = np.full((3, 2), -1)
    p = P.batch_plan([17, 16, 0], [0, 0, 0], table, [0, 1, 2], 2, 16, 64)
    assert list(p["lens"]) == [17, 0, 0] and p["count"] == 0 and p["errors"] == P.CAPACITY
    assert (p["slots"][17:33] == -1).all() and (p["seq_ids"][17:33] == 1).all()
    p = P.batch_plan([33, 1, 1], [0, 0, 15], table, [0, 1, 2], 3, 16, 64)  # the first has no columns, the last a page
    table[2, 0] = 1
    assert list(p["lens"]) == [0, 1, 16] and p["errors"] & P.CAPACITY


def test_fixed_rows():
    p = P.batch_plan([1, 0, 3, -1, 1], [15, 4, 0, 16, 16], np.array([[0], [1], [-1], [2], [3]]), [4, -1, -1, -1, -1], 1, 16, 10, 2)
    # the third has more tokens than rows, the last no column for its next page
    assert list(p["lens"]) == [16, 4, 0, 0, 16] and p["errors"] == P.CAPACITY and p["count"] == 2
    assert list(p["slots"]) == [15] + [-1] * 9 and list(p["offsets"]) == [0, 2, 4, 6, 8, 10]
    assert list(p["seq_ids"]) == [0, -1, -1, -1, 2, 2, -1, -1, 4, -1] and p["positions"][0] == 15


def test_rotations():
    x = np.random.default_rng(0).standard_normal((3, 2, 8))
    f, amp = R.frequencies(6)
    a = np.outer([0, 5, -7], f)
    for layout in ("half", "interleaved"):
        y = R.rotate(x, a, layout)
        np.testing.assert_array_equal(y[0], x[0])
        np.testing.assert_array_equal(y[..., 6:], x[..., 6:])
        np.testing.assert_allclose(np.square(y).sum(-1), np.square(x).sum(-1))
        np.testing.assert_allclose(R.rotate(y, -a, layout), x)
    y = R.rotate(x, a, "half")
    z = (x[1, 0, 0] + 1j * x[1, 0, 3]) * np.exp(5j * f[0])
    assert y[1, 0, 0] == pytest.approx(z.real) and y[1, 0, 3] == pytest.approx(z.imag)
    y = R.rotate(x, a, "interleaved")
    z = (x[2, 1, 2] + 1j * x[2, 1, 3]) * np.exp(-7j * f[1])
    assert y[2, 1, 2] == pytest.approx(z.real) and y[2, 1, 3] == pytest.approx(z.imag)
    assert amp == 1.0


@pytest.mark.parametrize("kw", [
    dict(), dict(base=500000.0), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
    dict(scaling="yarn", factor=32.0, base=150000.0, truncate=False), dict(scaling="yarn", factor=4.0),
    dict(scaling="yarn", factor=16.0, original_len=8192, low=1.5, high=20.0), dict(scaling="llama3", factor=8.0, original_len=8192),
    dict(scaling="llama3", factor=32.0, low=0.5, high=8.0, base=500000.0)])
@pytest.mark.parametrize("dim", [4, 64, 96, 128, 256])
def test_table(dim, kw):
    turns, amp = moe.moe_rope_table(dim, **kw)
    f, a = R.frequencies(dim, **kw)
    assert amp == pytest.approx(a, rel=1e-7)
    # a few roundings of 64-bit floats apart, and one step of the fraction
    np.testing.assert_allclose(turns.astype(np.float64) / 2.0 ** 64, f / (2 * math.pi), rtol=1e-13, atol=2.0 ** -63)
    own = moe.moe_rope_turns(f)
    np.testing.assert_allclose(own.astype(np.float64), turns.astype(np.float64), rtol=1e-13, atol=2.0)


def test_ends_of_the_scalings():
    """Fast pairs are kept, slow ones stretched in full."""
    plain, _ = R.frequencies(128)
    for scaling in ("yarn", "llama3"):
        f, _ = R.frequencies(128, scaling=scaling, factor=8.0)
        assert f[0] == plain[0] and f[-1] == pytest.approx(plain[-1] / 8)
    f, _ = R.frequencies(128, scaling="ntk", factor=8.0)
    assert f[0] == plain[0] and f[-1] == pytest.approx(plain[-1] / 8)


def test_turns_beyond_one_and_below_zero():
    t = moe.moe_rope_turns([2 * math.pi * 1.25, -2 * math.pi * 0.25, 0.0]).astype(np.float64) / 2.0 ** 64
    np.testing.assert_allclose(t, [0.25, 0.75, 0.0], atol=1e-15)


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=258), dict(rot_dim=64, base=1.0), dict(rot_dim=64, base=float("nan")),
    dict(rot_dim=64, scaling=7), dict(rot_dim=64, scaling="linear", factor=0.0), dict(rot_dim=64, scaling="yarn", original_len=0),
    dict(rot_dim=64, scaling="llama3", low=4.0, high=4.0), dict(rot_dim=2, scaling="ntk", factor=2.0),
    dict(rot_dim=64, amplitude=-1.0), dict(rot_dim=64, scaling="yarn", factor=float("inf"))])
def test_table_rejections(kw):
    with pytest.raises(moe.MoeError) as e:
        moe.moe_rope_table(**kw)
    assert e.value.code == 1


def test_turns_rejections():
    with pytest.raises(moe.MoeError):
        moe.moe_rope_turns([1.0, float("nan")])
    with pytest.raises(moe.MoeError):
        moe.rope(64, frequencies=np.ones(31), device="cpu")
