"""The rotation's cosines and sines by themselves, from pairs (1, 0) in fp32: angles of every fraction of a turn and far
positions, and their largest errors."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import bit_block_scaled_gb300 as moe
from gpu_helpers import built
from oracle import rope as R
from test_rope_turns import TWO_PI

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    return built()


def with_turns(turns, amplitude=1.0):
    """Rotary positions of given fractions of 2^64 of a turn."""
    r = moe.rope(2 * len(turns), "interleaved", frequencies=np.zeros(len(turns)), amplitude=amplitude)
    r.table.copy_(torch.from_numpy(np.array(turns, dtype=np.uint64).view(np.int64)))
    return r


def sines(r, pos):
    """(cosines, sines) [T, rot / 2] of an interleaved rotation, times its amplitude."""
    q = torch.zeros(len(pos), 1, r.rot_dim, device="cuda")
    q[..., 0::2] = 1
    moe.moe_rope(r, torch.tensor(pos, dtype=torch.int32, device="cuda"), q, q)
    return q[:, 0, 0::2].double().cpu().numpy(), q[:, 0, 1::2].double().cpu().numpy()


# Largest errors, amplitude 1: half a step of the result, 2^-25; in the larger of cosine and sine four roundings more of
# 2^-26 (1.49e-8) at most: the last coefficient's and its constant's times x^2 <= 1/16, and two of a value below 0.3; in the
# smaller four of 2^-28 (values below 1/8); series 2e-9. Then the angle's own error.
LARGE, SMALL = 2.0 ** -25 + 4 * 2.0 ** -26 + 1e-9, 2.0 ** -25 + 4 * 2.0 ** -28 + 2.5e-9
ANGLE = 2 * np.pi * 2.0 ** -33  # 2^31 steps of the table's 2^-65, and as much


def check(got, ref, angle=0.0):
    for g, r in zip(got, ref):
        assert (np.abs(g - r) <= np.where(np.abs(r) > 0.7, LARGE, SMALL) + angle).all()


def test_angles_between_the_steps_of_32_bits():
    """Fractions of a turn near every quarter that 32 bits do not hold."""
    rng = np.random.default_rng(0)
    turns = [(k << 62) + d for k in range(4) for d in (0.9 * 2 ** 32, 0.5 * 2 ** 32, 1.4 * 2 ** 32, 2 ** 20)]
    turns = [int(t) % 2 ** 64 for t in turns] + [(int(k) << 62) + int(d) & 2 ** 64 - 1 for k, d in
                                                 zip(rng.integers(0, 4, 48), rng.integers(-2 ** 35, 2 ** 35, 48))]
    turns += [int(t) for t in rng.integers(0, 2 ** 64, 64, dtype=np.uint64)]
    a = R.angles([1, -1], np.array(turns, dtype=object))
    c, s = sines(with_turns(turns), [1, -1])
    for got, ref in ((c, np.cos(a)), (s, np.sin(a))):
        # sines near 0 as small as they are: half a step of them, and 2^-34 turns
        near = np.abs(ref) < 2.0 ** -20
        assert near.any() and (np.abs(got - ref)[near] <= 2.0 ** -24 * np.abs(ref[near]) + 2 * np.pi * 2.0 ** -34 + 1e-15).all()
    check((c, s), (np.cos(a), np.sin(a)), 2 * np.pi * 2.0 ** -34)


@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_far_positions_of_a_frequency(base):
    """Against the frequencies as doubles, exactly: 2^31 - 1 positions turn the fastest pair 340 million times."""
    pos = [2 ** 31 - 1, -2 ** 31, 10 ** 9 + 7, 131072, 1]
    f, _ = R.frequencies(64, base=base)
    ref = np.array([[float(Fraction(float(x)) * p % TWO_PI) for x in f] for p in pos])
    r = moe.rope(64, "interleaved", frequencies=f)
    check(sines(r, pos), (np.cos(ref), np.sin(ref)), ANGLE)
    plain = moe.rope(64, "interleaved", base=base)
    assert np.abs(plain.table.cpu().numpy() - r.table.cpu().numpy()).max() <= 2 ** 12  # a last bit of the double or two
