"""moe_fp4_linear in every kernel and tile (tests/test_front_sizes.py holds the sizes to them): output types, rows off the
16-byte grid and columns that no bulk copy writes, one scale for all weights, rows that hold no number."""
import pytest
import torch

from gpu_helpers import built
from test_front_sizes import PRODUCTS
from test_gpu_fp4 import FMTS, TYPES, check_linear, rows

pytestmark = pytest.mark.gpu
# rows as wide as N, off the 16-byte grid; wider, on it, so that the last columns are written one by one; wider, off it
PADS = {"as_they_are": lambda N: N, "on_the_grid": lambda N: (N + 7) // 8 * 8 + 8, "off_the_grid": lambda N: N + 3}
SIZES = [s for kernel in PRODUCTS for s in PRODUCTS[kernel]]
WIDE = PRODUCTS["wide", 256, False]


@pytest.fixture(scope="module", autouse=True)
def lib():
    return built()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,N,K", [s for s in SIZES if s not in WIDE])
def test_narrow(T, N, K, fmt):
    for i, (dtype, pad) in enumerate(zip(TYPES, PADS.values())):
        check_linear(T, N, K, fmt, dtype, i != 1, T + i, 0.37 if fmt == "nvfp4" and i == 2 else None, pad(N))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad", PADS)
@pytest.mark.parametrize("T,N,K", WIDE)
def test_wide(T, N, K, pad, dtype, fmt):
    one_scale = fmt == "nvfp4" and pad == "as_they_are"
    check_linear(T, N, K, fmt, dtype, pad != "off_the_grid", T, 0.0037 if one_scale else None, PADS[pad](N))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,N,K", [PRODUCTS[k][0] for k in PRODUCTS if PRODUCTS[k][0][0] > 4])
def test_rows_that_hold_no_numbers(T, N, K, fmt):
    """A NaN or an infinity makes its token's outputs NaN and no other's, in the first tile and in the last."""
    x = rows(T, K, torch.bfloat16, T)
    x[0] = 0
    x[1, 5], x[T - 1, K - 1] = float("inf"), float("nan")
    x[2], x[3] = 1e30, 1e-38
    out = check_linear(T, N, K, fmt, "bf16", True, x=x)
    bad = torch.isnan(out)
    assert bad[1].all() and bad[T - 1].all() and bad.any(dim=1).sum() == 2
