"""The sizes with which the GPU tests of the 4-bit product and of rotary positions reach a kernel, a tile, a split of K or
several rows a lane: held to them here, over a runtime that launches nothing (fake_cuda.py), so that a changed rule of
choice does not leave one of them without a test. And the grids of the most tokens that the calls take."""
import re

import pytest

import bit_block_scaled_gb300 as moe
from fake_cuda import Library, link

P = 1 << 20  # stands for every pointer; nothing is read

# (kernel, tokens a tile, whether K is split): sizes (T, N, K). "wide" is the kernel of pairs of CTAs.
PRODUCTS = {
    ("narrow", 16, False): [(1, 130, 64), (13, 130, 96)],
    ("narrow", 16, True): [(1, 5120, 2880), (16, 640, 4096)],
    ("narrow", 32, False): [(20, 333, 544)],
    ("narrow", 32, True): [(20, 640, 2880)],
    ("narrow", 64, False): [(900, 333, 608)],
    ("narrow", 64, True): [(40, 1000, 2880)],
    ("narrow", 128, False): [(256, 5120, 544), (400, 2880, 1024)],
    ("narrow", 128, True): [(493, 890, 5984)],
    ("wide", 256, False): [(3000, 2885, 608), (9000, 333, 608)],
}
# (T, kv heads, head_dim): four rows of keys and values a lane
WRITES = [(6700, 3, 256), (13001, 3, 128), (16001, 5, 64)]
# (T, q heads, k heads, head_dim, rot): 16 tokens a CTA
ROTATIONS = [(10007, 2, 1, 64, 64), (10007, 2, 1, 64, 40), (10007, 1, 1, 80, 64)]


@pytest.fixture(scope="module")
def path(tmp_path_factory):
    return link(tmp_path_factory.mktemp("fake"))


@pytest.fixture
def lib(path, tmp_path):
    l = Library(path, tmp_path)
    l.lib.fake_encoder(1)
    return l


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("kernel", PRODUCTS)
def test_products(lib, kernel, fmt):
    for T, N, K in PRODUCTS[kernel]:
        for dtype in (0, 1, 2):
            r = P if fmt == 0 else None
            x, w = moe.Fp4(fmt, T, K, 1, P, P, r), moe.Fp4(fmt, N, K, 1, P, P, r)
            assert lib.lib.moe_fp4_linear(x, w, None, P, dtype, N, P, None) == 0
            (name, _, grid, _, cluster), = lib.launches()
            if kernel[0] == "wide":
                assert f"wide_kernelILi{fmt}ELi{dtype}E" in name, (T, N, K, name)
                continue
            assert f"narrow_kernelILi{fmt}ELi{kernel[1]}E" in name and (cluster > 1) == kernel[2], (T, N, K, name, cluster)
            assert grid[0] == -(-T // kernel[1]) * -(-N // 128) * cluster


def write_grid(lib, T, hk, D, q=None, q_heads=0):
    r, c = moe.Rope(D, 0, 1.0, P), moe.KvCache(2, 1000, 16, hk, D, P)
    args = [P, hk * D, D, P, hk * D, D, 0, P, T, c, P, None]
    assert lib.lib.moe_rope_kv_write(r, P, q, q_heads * D, D, q_heads, q, q_heads * D, D, *args) == 0
    return lib.launches()[0][2][0]


@pytest.mark.parametrize("T,hk,D", WRITES)
def test_writes(lib, T, hk, D):
    per = 256 // (D // 8)
    assert write_grid(lib, T, hk, D) == -(-T * hk // (4 * per))  # four rows a lane
    assert T * hk % (4 * per) and hk * 4 % per  # a ragged end, and tokens that end within a lane's walk
    assert write_grid(lib, 700, hk, D) == -(-700 * hk // per)


def rope_grid(lib, T, hq, hk, D, rot):
    k = (P, hk * D, D, hk, P + (1 << 29), hk * D, D)
    assert lib.lib.moe_rope(moe.Rope(rot, 0, 1.0, P), P, T, D, P, hq * D, D, hq, P + (1 << 30), hq * D, D, *k, 0, None) == 0
    return lib.launches()[0][2][0]


@pytest.mark.parametrize("T,hq,hk,D,rot", ROTATIONS)
def test_rotations(lib, T, hq, hk, D, rot):
    assert rope_grid(lib, T, hq, hk, D, rot) == -(-T // 16)


@pytest.mark.parametrize("T", [2 ** 31 - 1, 2 ** 31 - 16, 2 ** 31 - 17])
def test_the_most_tokens(lib, T):
    """One head of two columns: 16 tokens a CTA, the last of them within 16 of 2^31."""
    assert rope_grid(lib, T, 1, 0, 2, 2) == -(-T // 16)
    assert write_grid(lib, T, 1, 64, P, 1) == -(-T // 16) + -(-T // 32)  # queries, and a row of keys a lane
