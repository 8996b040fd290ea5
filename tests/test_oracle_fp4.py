"""Pins of oracle/fp4.py: closed forms, brute force, and the tiles."""
import numpy as np
import pytest

from oracle import fp4 as F
from oracle.formats import E2M1_VALUES, E4M3_VALUES


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_values_that_fit_come_back(fmt):
    rng = np.random.default_rng(0)
    block = F.BLOCK[fmt]
    codes = rng.integers(0, 16, (6, 96))
    codes[:, ::block] = 7  # a block's largest magnitude is 6
    s = 2.0 ** rng.integers(-3, 4, (6, 96 // block))
    if fmt == "nvfp4":
        s[:, 0] = 256.0
    x = E2M1_VALUES[codes] * np.repeat(s, block, axis=1)
    q, sc, r = F.quantise_rows(x, fmt)
    np.testing.assert_array_equal(F.values(q, sc, r, fmt), x)


def test_nearest_of_all():
    """Each code is the nearest of all 16 to x over its scales, and the scales are the least that fit."""
    x = np.random.default_rng(1).standard_normal((5, 64)) * 10
    q, sc, r = F.quantise_rows(x, "nvfp4")
    amax = np.abs(x).max(axis=1)
    assert np.all(amax / r <= 2688) and np.all(amax / (r / 2) > 2688)
    back = F.values(q, sc, r, "nvfp4")
    s = np.repeat(E4M3_VALUES[sc], 16, axis=1) * r[:, None]
    best = np.abs(np.abs(x)[..., None] - E2M1_VALUES[:8] * s[..., None]).min(axis=-1)
    np.testing.assert_allclose(np.abs(x - back), best, rtol=1e-12)
    q, sc, _ = F.quantise_rows(x, "mxfp4")
    s = 2.0 ** (sc.astype(float) - 127)
    b = np.abs(x.reshape(5, 2, 32)).max(axis=2)
    assert np.all(b / s <= 6) and np.all(b / (s / 2) > 6)


@pytest.mark.parametrize("rows,blocks", [(1, 1), (127, 4), (128, 5), (300, 23)])
def test_tiles(rows, blocks):
    s = np.random.default_rng(2).integers(1, 256, (rows, blocks)).astype(np.uint8)
    t = F.tile(s)
    assert t.size == -(-rows // 128) * -(-blocks // 4) * 512
    for r, b in [(0, 0), (rows - 1, blocks - 1), (rows // 2, blocks // 2)]:
        at = ((r // 128) * -(-blocks // 4) + b // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4
        assert t[at] == s[r, b]
    np.testing.assert_array_equal(F.untile(t, rows, blocks), s)


def test_linear_by_loops():
    rng = np.random.default_rng(3)
    x, w, b = rng.standard_normal((2, 32)), rng.standard_normal((3, 32)), rng.standard_normal(3)
    out, mag = F.linear(x, w, b)
    for t in range(2):
        for n in range(3):
            assert out[t, n] == pytest.approx(sum(x[t, k] * w[n, k] for k in range(32)) + b[n])
            assert mag[t, n] == pytest.approx(sum(abs(x[t, k] * w[n, k]) for k in range(32)))


def test_no_numbers():
    x = np.full((2, 64), 6.0)  # a scale of E4M3 times 6, and of E8M0
    x[0, 40] = np.inf
    v = F.values(*F.quantise_rows(x, "nvfp4"), "nvfp4")
    assert np.isnan(v[0]).all() and (v[1] == 6).all()
    v = F.values(*F.quantise_rows(x, "mxfp4"), "mxfp4")
    assert np.isnan(v[0, 32:]).all() and (v[0, :32] == 6).all()
