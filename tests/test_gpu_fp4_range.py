"""moe_fp4_linear over the whole range of values: row scales whose product with a sum leaves fp32's range although the
result does not. In every kernel and tile (tests/test_front_sizes.py holds the sizes to them)."""
import numpy as np
import pytest
import torch

import bit_block_scaled_gb300 as moe
from gpu_helpers import built, ws_status
from oracle import fp4 as F
from test_front_sizes import PRODUCTS
from test_gpu_fp4 import TYPES, f64, operand

pytestmark = pytest.mark.gpu
SIZES = [PRODUCTS[k][0] for k in PRODUCTS]
# powers of two about which a row's values lie; all of a token's products with weights of the opposite one are numbers
FAR = (0, 117, -120, 100, -100, 71, 72, -49, -50, 30, -30, 64)


@pytest.fixture(scope="module", autouse=True)
def lib():
    return built()


def spread(T, K, seed, shift=0):
    """Rows of values about 2^e, e from FAR in turn, the last one zeros."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=g, dtype=torch.float64)
    e = torch.tensor([FAR[(i + shift) % len(FAR)] for i in range(T)], dtype=torch.float64)
    x = (x * 2.0 ** e[:, None]).float()
    if T > 1:
        x[-1] = 0
    return x.cuda()


def quantised(x, fmt="nvfp4"):
    b, m = operand(*x.shape, fmt)
    moe.moe_fp4_quantize(x, m)
    return b, m


def values(x, fmt="nvfp4"):
    return F.values(*F.quantise_rows(f64(x), fmt), fmt)


def product(xm, wm, bias, t):
    out, ws = torch.zeros(xm.rows, wm.rows, dtype=t, device="cuda"), ws_status()
    moe.moe_fp4_linear(xm, wm, bias, out, ws)
    assert moe.moe_read_status(ws) == 0
    return out


def check(got, xv, wv, bias=None):
    """As in test_gpu_fp4.check_linear, and half a step of the type's smallest numbers."""
    t, K = got.dtype, xv.shape[1]
    ref, mag = F.linear(xv, wv, None if bias is None else f64(bias))
    tol = torch.finfo(t).eps / 2 * (np.abs(ref) + torch.finfo(t).tiny) + (K / 64 + 4) * 2.0 ** -22 * (mag + np.abs(ref))
    got = f64(got)
    assert not np.isnan(got).any()
    top = float(torch.finfo(t).max) * (1 + torch.finfo(t).eps / 4)
    over = np.isinf(got)
    assert (np.sign(got[over]) * ref[over] >= top - tol[over]).all()
    err = np.abs(got - ref)
    assert (err[~over] <= tol[~over]).all(), np.nanmax(err[~over] / tol[~over])
    return ref


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T,N,K", SIZES)
def test_rows_of_every_size(T, N, K, dtype):
    t = TYPES[dtype]
    for shift in ((0, 1, 2) if T == 1 else (0,)):
        x, w = spread(T, K, T, shift), spread(N, K, N + 1, 2)
        _, xm = quantised(x)
        _, wm = quantised(w)
        ref = check(product(xm, wm, None, t), values(x), values(w))
        bias = torch.randn(N, device="cuda").to(t)
        check(product(xm, wm, bias, t), values(x), values(w), bias)
        top = float(torch.finfo(t).max)
        assert T == 1 or ((np.abs(ref) > 2 * top).any() and (np.abs(ref[:, 0]) > 0).any())  # there is something to see


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,N,K", SIZES)
def test_large_tokens_with_small_weights(T, N, K, fmt):
    """1e36 throughout by 1e-3 throughout: a number in bf16, and so is its sum."""
    x, w = torch.full((T, K), 1e36, device="cuda"), torch.full((N, K), 1e-3, device="cuda")
    _, xm = quantised(x, fmt)
    _, wm = quantised(w, fmt)
    got = product(xm, wm, None, torch.bfloat16)
    assert torch.isfinite(got).all()
    check(got, values(x[:1], fmt).repeat(T, 0), values(w[:1], fmt).repeat(N, 0))


@pytest.mark.parametrize("T,N,K", SIZES)
def test_small_tokens_with_large_weights(T, N, K):
    """Subnormal tokens by the small values of weights that have a large one: a sum times the token's scale has few bits left."""
    g = torch.Generator().manual_seed(K)
    x, w = torch.zeros(T, K), torch.randn(N, K, generator=g) * 2.0 ** 103
    x[:, 16:] = torch.randint(-6, 7, (T, K - 16), generator=g).float() * 2.0 ** -133
    w[:, 0] = 2.0 ** 120
    x, w = x.cuda(), w.cuda()
    _, xm = quantised(x)
    _, wm = quantised(w)
    check(product(xm, wm, None, torch.float32), values(x), values(w))


@pytest.mark.parametrize("T,N,K", [s for s in SIZES if s[0] > 1])
def test_rows_do_not_depend_on_their_neighbours(T, N, K):
    """Bit for bit, whatever the sizes of the tile's other rows."""
    x, w = spread(T, K, 1), spread(N, K, 2, 3)
    calm = x.clone()
    ordinary = torch.tensor([FAR[i % len(FAR)] in (0, 30, -30, 64) for i in range(T)])
    calm[~ordinary.cuda()] = 1.0
    _, wm = quantised(w)
    a, b = (product(quantised(y)[1], wm, None, torch.float32) for y in (x, calm))
    assert torch.equal(a[ordinary.cuda()][:-1], b[ordinary.cuda()][:-1])


@pytest.mark.parametrize("T,N,K", SIZES)
def test_row_scales_of_the_callers(T, N, K):
    """Scales of any sign and size, no powers of two; one for all weights; NaN and infinity stay what they are."""
    x, w = spread(T, K, 5), torch.randn(N, K, device="cuda")
    (xq, xs, _), _ = quantised(x)
    (wq, wsc, _), _ = quantised(w)
    g = torch.Generator().manual_seed(T)
    xr = (torch.randn(T, generator=g) * 2.0 ** torch.randint(-126, 100, (T,), generator=g)).cuda()
    for wr in (torch.full((1,), -3.7e-30, device="cuda"), torch.full((1,), 1.3e25, device="cuda")):
        got = product(moe.fp4(xq, xs, "nvfp4", xr), moe.fp4(wq, wsc, "nvfp4", wr), None, torch.float32)
        xv = F.values(xq.cpu().numpy(), F.untile(xs.cpu().numpy(), T, K // 16), f64(xr), "nvfp4")
        wv = F.values(wq.cpu().numpy(), F.untile(wsc.cpu().numpy(), N, K // 16), f64(wr), "nvfp4")
        check(got, xv, wv)
    wr = torch.ones(N, device="cuda")
    wr[0], wr[N - 1] = float("inf"), float("nan")
    xr[T - 1] = 2.0 ** 100
    got = product(moe.fp4(xq, xs, "nvfp4", xr), moe.fp4(wq, wsc, "nvfp4", wr), None, torch.float32)
    assert torch.isnan(got[:, N - 1]).all() and not torch.isfinite(got[:, 0]).any()
    assert not torch.isnan(got[:, 1:N - 1]).any()
