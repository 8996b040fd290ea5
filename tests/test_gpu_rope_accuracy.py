"""The rotation's cosines and sines by themselves, from pairs (1, 0) in fp32: angles of every fraction of a turn and far
positions, their largest and root mean square errors, and what is left of them in quantised keys."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import bit_block_scaled_gb300 as moe
from gpu_helpers import built, ws_status
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


# Root mean square errors of the same arithmetic, step by step in fp32 (numpy): 1.94e-8 and 1.15e-8 of the amplitude at
# 1, 2.67e-8 and 1.00e-8 at YaRN's for a factor of 32 (1.3466), where results above 1 have steps twice as long. Correct
# rounding: 1.72e-8 and 1.13e-8, 2.49e-8 and 0.98e-8. The bounds are 2% above; 1.3 million values give it to 0.1%.
@pytest.mark.parametrize("kw,large,small", [(dict(), 1.98e-8, 1.18e-8),
                                            (dict(scaling="yarn", factor=32.0), 2.72e-8, 1.02e-8)])
def test_root_mean_square(kw, large, small):
    r = moe.rope(128, "interleaved", **kw)
    pos = np.random.default_rng(1).integers(-2 ** 31, 2 ** 31, 20000)
    with np.errstate(over="ignore"):
        a = (r.table.cpu().numpy()[None, :] * pos[:, None].astype(np.int64)).astype(np.float64) * (2 * np.pi / 2.0 ** 64)
    a = np.where(np.abs(a) > 1e-3, a, 0)  # what is next to 0 would add little
    got, ref = sines(r, pos.tolist()), (r.amplitude * np.cos(a), r.amplitude * np.sin(a))
    e = np.stack([g - x for g, x in zip(got, ref)])[:, a != 0] / r.amplitude
    big = (np.abs(np.stack(ref)) > r.amplitude * np.sqrt(0.5))[:, a != 0]
    assert np.sqrt(np.mean(e[big] ** 2)) <= large and np.sqrt(np.mean(e[~big] ** 2)) <= small


def e4m3(x):
    """The nearest of E4M3's numbers, ties to even; |x| <= 448."""
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -20))), -6) - 3)
    return np.rint(x / step) * step


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_quantised_keys(layout):
    """Keys in an FP8 cache are codes of a value next to the 64-bit one, and nearly all those of the 64-bit one itself: of
    some 50 million rotated so, step by step in numpy, 64 were not (76 with every step rounded as elementary fp32
    operations round, from sines of 64 bits), so of one million 1.3; more than 12 come once in 10^8."""
    T, H, D = 2000, 4, 128
    g = torch.Generator().manual_seed(3)
    k = torch.randn(T, H, D, generator=g)
    k[..., ::16] *= 8
    k = k.bfloat16().cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    r = moe.rope(D, layout)
    data = torch.zeros(T // 16, H, 1, moe.moe_kv_record_bytes("fp8", D), dtype=torch.uint8, device="cuda")
    c, ws = moe.kv_cache(data, "fp8", D), ws_status()
    moe.moe_rope_kv_write(r, pos, None, None, k, k, pos, c, ws)
    got, v = torch.empty(T, H, D, device="cuda"), torch.empty(T, H, D, device="cuda")
    moe.moe_kv_read(c, pos, got, v, ws)
    x = k.double().cpu().numpy()
    ref = R.rotate(x, R.angles(range(T), r.table.cpu().numpy().view(np.uint64)), layout)
    top = np.abs(ref).max(-1, keepdims=True) / 448
    m, e = np.frexp(top)
    scale = 2.0 ** np.where(m == 0.5, e - 1, e)
    clear = np.abs(top / scale - 1).squeeze(-1) > 2.0 ** -20  # the row's exponent is decided
    clear &= np.abs(top / scale - 0.5).squeeze(-1) > 2.0 ** -20
    # a product and a sum, half a step each, and the sines' errors, of the pair's magnitudes
    near = 2.0 ** -24 * np.abs(ref) + (2.0 ** -24 + LARGE + SMALL) * np.abs(x).max(-1, keepdims=True) * 2
    got = got.double().cpu().numpy()
    ok = (got >= e4m3((ref - near) / scale) * scale) & (got <= e4m3((ref + near) / scale) * scale)
    assert clear.mean() > 0.999 and ok[clear].all()
    assert (got != e4m3(ref / scale) * scale)[clear].sum() <= 12
