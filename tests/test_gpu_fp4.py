"""4-bit operands on the GPU: quantisation byte by byte against the oracle, the tiles of the scales, and the product
against 64 bits."""
import numpy as np
import pytest
import torch

import bit_block_scaled_gb300 as moe
from gpu_helpers import built, ws_status
from oracle import fp4 as F

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FMTS = ("nvfp4", "mxfp4")


@pytest.fixture(scope="module", autouse=True)
def lib():
    return built()


def f64(t):
    return t.double().cpu().numpy()


def operand(T, K, fmt, fill=0xAB):
    """Buffers of a 4-bit matrix, not zeroed, and the matrix."""
    q = torch.full((T, K // 2), fill, dtype=torch.uint8, device="cuda")
    s = torch.full((moe.moe_fp4_scale_bytes(fmt, T, K),), fill, dtype=torch.uint8, device="cuda")
    r = torch.full((T,), 3.0, device="cuda") if fmt == "nvfp4" else None
    return (q, s, r), moe.fp4(q, s, fmt, r)


def rows(T, K, dtype, seed=0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=g) * torch.exp(spread * torch.randn(T, 1, generator=g))
    x[:, ::37] *= 20
    return x.to(dtype).cuda()


def check_quantised(x, fmt):
    T, K = x.shape
    (q, s, r), m = operand(T, K, fmt)
    moe.moe_fp4_quantize(x, m)
    eq, es, er = F.quantise_rows(f64(x), fmt)
    assert np.array_equal(q.cpu().numpy(), eq)
    got = F.untile(s.cpu().numpy(), T, K // F.BLOCK[fmt])
    assert np.array_equal(got, es)
    if K // F.BLOCK[fmt] % 4:  # scales past the row are 0
        wide = -(-(K // F.BLOCK[fmt]) // 4) * 4
        assert not F.untile(s.cpu().numpy(), T, wide)[:, K // F.BLOCK[fmt]:].any()
    if er is not None:
        np.testing.assert_array_equal(f64(r), er)
    return (q, s, r), m


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K", [(1, 32), (1, 2880), (3, 64), (5, 96), (7, 16384), (64, 2880), (129, 512), (200, 1056),
                                 (700, 2880), (650, 8192), (2, 32768), (613, 32), (609, 4096)])
def test_quantize(fmt, dtype, T, K):
    check_quantised(rows(T, K, TYPES[dtype], seed=T + K), fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_ties_and_extremes(fmt, dtype):
    """Every tie of E2M1 under every block scale, the ends of the exponents, zeros, and rows that hold no number."""
    t = TYPES[dtype]
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -0.0])
    blocks = []
    for m in range(8, 16):  # significands of E4M3; the row's scale is 1 or a power of two
        blocks += [ties * (m / 8.0) * 2.0 ** k for k in (-3, 0, 3)]
    x = torch.cat(blocks).view(1, -1)
    x = torch.cat((x, x, torch.zeros(1, 2 * x.shape[1] % 32)), 1) if (2 * x.shape[1]) % 32 else torch.cat((x, x), 1)
    x[0, 16] = 448.0 * 6  # pins the row scale at 1
    K = x.shape[1]
    top = float(torch.finfo(t).max)
    many = [x, torch.zeros(1, K), -x, x * 2.0 ** -10, torch.full((1, K), top), torch.full((1, K), -top)]
    tiny = torch.zeros(1, K)
    tiny[0, 5] = torch.finfo(t).tiny if dtype != "bf16" else 2.0 ** -126
    many.append(tiny)
    small = torch.zeros(1, K)
    small[0, :16] = 2.0 ** -24 if dtype == "fp16" else 2.0 ** -130
    many.append(small)
    for bad in (float("nan"), float("inf"), -float("inf")):
        y = x.clone()
        y[0, 77] = bad
        many.append(y)
    check_quantised(torch.cat(many).to(t).cuda(), fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_strided_rows(fmt):
    big = rows(50, 4096, torch.bfloat16)
    check_quantised(big[:, 1024:1024 + 2880], fmt)
    check_quantised(big[::3, 8:8 + 96], fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K", [(1, 32), (130, 2880), (33, 96)])
def test_dequantize(fmt, dtype, T, K):
    x = rows(T, K, torch.bfloat16, seed=K)
    x[T // 2, 3] = float("nan")
    bufs, m = operand(T, K, fmt)
    moe.moe_fp4_quantize(x, m)
    out = torch.full((T, K + 8), 7.0, dtype=TYPES[dtype], device="cuda")
    moe.moe_fp4_dequantize(m, out[:, :K])
    ref = F.values(*F.quantise_rows(f64(x), fmt), fmt)
    np.testing.assert_array_equal(f64(out[:, :K]), f64(torch.from_numpy(ref).to(TYPES[dtype])))
    assert (out[:, K:] == 7).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("N,K", [(1, 32), (130, 2880), (300, 96)])
def test_pack_scales(fmt, N, K):
    plain = torch.randint(0, 256, (N, K // F.BLOCK[fmt]), dtype=torch.uint8, device="cuda")
    out = torch.full((moe.moe_fp4_scale_bytes(fmt, N, K),), 0x77, dtype=torch.uint8, device="cuda")
    moe.moe_fp4_pack_scales(plain, fmt, K, out)
    wide = -(-plain.shape[1] // 4) * 4
    got = F.untile(out.cpu().numpy(), N, wide)
    assert np.array_equal(got[:, :plain.shape[1]], plain.cpu().numpy()) and not got[:, plain.shape[1]:].any()


def check_linear(T, N, K, fmt, dtype, bias, seed=0, gscale=None, ldo=None, x=None):
    t = TYPES[dtype]
    x = rows(T, K, torch.bfloat16, seed) if x is None else x
    w = rows(N, K, torch.bfloat16, seed + 1, 0.3) * K ** -0.5
    (_, _, _), xm = bx = operand(T, K, fmt)
    (wq, wsc, wr), wm = bw = operand(N, K, fmt)
    moe.moe_fp4_quantize(x, xm)
    moe.moe_fp4_quantize(w, wm)
    if gscale:  # one scale for all rows, as in a checkpoint
        wr = torch.tensor([gscale], device="cuda")
        wm = moe.fp4(wq, wsc, fmt, wr)
    b = torch.randn(N, device="cuda").to(t) if bias else None
    ldo = N if ldo is None else ldo
    buf = torch.full((T, ldo), 9.0, dtype=t, device="cuda")
    ws = ws_status()
    moe.moe_fp4_linear(xm, wm, b, buf[:, :N], ws)
    torch.cuda.synchronize()
    assert moe.moe_read_status(ws) == 0
    xq, xs, xr = F.quantise_rows(f64(x), fmt)
    xv = F.values(xq, xs, xr, fmt)
    wv = F.values(wq.cpu().numpy(), F.untile(wsc.cpu().numpy(), N, K // F.BLOCK[fmt]), None if wr is None else f64(wr), fmt)
    ref, mag = F.linear(xv, wv, None if b is None else f64(b))
    got = f64(buf[:, :N])
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    # half a step of the output, and of the sums: each of the K / 64 additions, the row scales and the bias, off by
    # 2^-22 of all magnitudes at most (sums may be cut, not rounded)
    tol = torch.finfo(t).eps / 2 * np.abs(ref) + (K / 64 + 4) * 2.0 ** -22 * (mag + np.abs(ref)) + 1e-30
    # from half a step past the largest number on, a type has infinity
    top = float(torch.finfo(t).max) * (1 + torch.finfo(t).eps / 4)
    over = np.isinf(got)
    assert (np.sign(got[over]) * ref[over] >= top - tol[over]).all()
    ok = ~np.isnan(ref) & ~over
    err = np.abs(got - ref)
    assert (err[ok] <= tol[ok]).all(), (err[ok] / tol[ok]).max()
    assert (buf[:, N:] == 9).all()
    return buf[:, :N]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,N,K", [(1, 128, 64), (1, 128, 32), (1, 1, 32), (1, 5120, 2880), (3, 200, 96), (16, 256, 256),
                                   (17, 333, 544), (40, 1000, 2880), (100, 2688, 4096), (128, 128, 1024), (129, 136, 800)])
def test_linear(fmt, T, N, K):
    check_linear(T, N, K, fmt, "bf16", True, seed=T)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bias", [False, True])
def test_linear_types(fmt, dtype, bias):
    check_linear(5, 200, 576, fmt, dtype, bias, ldo=203)
    check_linear(150, 72, 2880, fmt, dtype, bias, gscale=0.37 if fmt == "nvfp4" else None)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,N,K", [(512, 192, 256), (513, 200, 96), (600, 1, 32), (1000, 1000, 544), (1111, 5120, 2880),
                                   (4096, 3000, 1600), (700, 8200, 4096)])
def test_linear_many_tokens(fmt, T, N, K):
    check_linear(T, N, K, fmt, "bf16", True, seed=T)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,ldo", [(384, 384), (333, 333), (333, 400), (40, 41)])
def test_linear_many_tokens_types(fmt, dtype, N, ldo):
    check_linear(900, N, 608, fmt, dtype, True, ldo=ldo, gscale=0.0037 if fmt == "nvfp4" else None)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [3, 40, 150, 600])
def test_linear_rows_that_hold_no_numbers(fmt, T):
    """A NaN or an infinity makes its token's outputs NaN and no other's; rows of zeros and of extremes are as they are."""
    x = rows(T, 320, torch.bfloat16, T)
    x[1, 5] = float("inf")
    x[T - 1, 319] = float("nan")
    x[0] = 0
    if T > 3:
        x[2] = 1e30
        x[3] = 1e-38
    out = check_linear(T, 200, 320, fmt, "bf16", True, x=x)
    assert torch.isnan(out[1]).all() and torch.isnan(out[T - 1]).all() and torch.isnan(out).any(dim=1).sum() == 2


def test_linear_weights_without_numbers():
    """An MXFP4 block of exponent 255 makes its output column NaN, and no other."""
    x, w = rows(20, 128, torch.bfloat16), rows(130, 128, torch.bfloat16, 1)
    w[129, 70] = float("nan")
    (_, xm), (_, wm) = operand(20, 128, "mxfp4"), operand(130, 128, "mxfp4")
    moe.moe_fp4_quantize(x, xm)
    moe.moe_fp4_quantize(w, wm)
    out = torch.zeros(20, 130, device="cuda")
    moe.moe_fp4_linear(xm, wm, None, out, ws_status())
    assert torch.isnan(out[:, 129]).all() and not torch.isnan(out[:, :129]).any()


@pytest.mark.parametrize("T,N,K", [(1, 640, 2880), (24, 640, 2880), (100, 640, 8192), (333, 2880, 1024), (2000, 1500, 2880)])
def test_linear_repeats_itself_and_is_captured(T, N, K):
    """Bit for bit, on another stream and in a graph whose inputs change."""
    x, w = rows(T, K, torch.bfloat16), rows(N, K, torch.bfloat16, 1)
    (bx, xm), (_, wm) = operand(T, K, "nvfp4"), operand(N, K, "nvfp4")
    moe.moe_fp4_quantize(w, wm)
    moe.moe_fp4_quantize(x, xm)
    ws = ws_status()
    a, b = torch.zeros(T, N, device="cuda"), torch.zeros(T, N, device="cuda")
    moe.moe_fp4_linear(xm, wm, None, a, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        moe.moe_fp4_linear(xm, wm, None, b, ws)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    g, y = torch.cuda.CUDAGraph(), x.clone()
    with torch.cuda.graph(g, stream=s):
        moe.moe_fp4_quantize(y, xm)
        moe.moe_fp4_linear(xm, wm, None, b, ws)
    b.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    y.copy_(x.flip(0))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(b, a.flip(0)) and moe.moe_read_status(ws) == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_a_part_of_the_rows(fmt):
    """Operands over the first rows of larger buffers, as a padded batch has: what lies behind stays, in the output too."""
    T, N, K, most = 70, 130, 96, 300
    q = torch.full((most, K // 2), 0xFF, dtype=torch.uint8, device="cuda")
    s = torch.full((moe.moe_fp4_scale_bytes(fmt, most, K),), 0xFF, dtype=torch.uint8, device="cuda")  # NaN to both formats
    r = torch.full((most,), float("nan"), device="cuda") if fmt == "nvfp4" else None
    xm = moe.fp4(q[:T], s[:moe.moe_fp4_scale_bytes(fmt, T, K)], fmt, None if r is None else r[:T])
    x, w = rows(T, K, torch.bfloat16), rows(N, K, torch.bfloat16, 1)
    (wq, wsc, wr), wm = operand(N, K, fmt)
    moe.moe_fp4_quantize(x, xm)
    moe.moe_fp4_quantize(w, wm)
    out = torch.full((most, N), 5.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_fp4_linear(xm, wm, None, out[:T], ws_status())
    assert (out[T:] == 5).all() and (q[T:] == 0xFF).all()
    ref, mag = F.linear(F.values(*F.quantise_rows(f64(x), fmt), fmt), F.values(*F.quantise_rows(f64(w), fmt), fmt))
    assert (np.abs(f64(out[:T]) - ref) <= 2.0 ** -8 * np.abs(ref) + 6 * 2.0 ** -22 * mag).all()
