"""moe_residual_norm against the float64 oracle.

fp32 arithmetic: a row sum over at most 32 terms a thread, five joins in a warp and five over the warps is off by at
most 42 * 2^-24 of the sum of magnitudes; with the roundings of the products that follow, an element of a norm is off
by at most 64 * 2^-24 of the largest term of its row ((|x| + |mean|) / sd * |w| + |b|), each of the two norms adding
that. Then one rounding to the output's type (half a step, eps / 2)."""
import numpy as np
import pytest
import torch

import bit_block_scaled_gb300 as moe
from gpu_helpers import built
from oracle import seam as S

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

#: the smallest positive value of each type
SMALLEST = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}


@pytest.fixture(scope="module", autouse=True)
def lib():
    return built()


def rnd(*shape, dtype="fp32", seed=0, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(TYPES[dtype]).cuda()


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def spec(kind, H, seed, wtype="fp32", **kw):
    if kind is None:
        return None, None
    w = (1 + rnd(H, seed=seed, std=0.2)).to(TYPES[wtype])
    b = rnd(H, seed=seed + 1, std=0.2).to(TYPES[wtype]) if kind == "layer" else None
    keep = moe.norm(kind, w, b, **kw)
    keep.tensors = (w, b)
    return keep, dict(kind=kind, weight=f64(w), bias=f64(b), **kw)


def terms(x, s):
    """Largest term of each row of a norm's sum."""
    if s is None:
        return np.abs(x).max(axis=1, keepdims=True)
    _, r = S.norm(x, **s)
    w = 1.0 if s.get("weight") is None else np.abs(s["weight"] + s.get("offset", 0.0))
    b = 0.0 if s.get("bias") is None else np.abs(s["bias"])
    mean = np.abs(x).mean(axis=1, keepdims=True)
    return ((np.abs(x) + mean) * r * w + b).max(axis=1, keepdims=True)


def half(t):
    return torch.finfo(t.dtype).eps / 2


def run(T, H, act="bf16", res="bf16", gate=None, post="rms", pre="rms", alpha=1.0, wtype="fp32", has_res=True,
        write_h=True, mean=0.0, stream=None, **kw):
    z = rnd(T, H, dtype=act, seed=1, std=2.0) + mean
    r = rnd(T, H, dtype=res, seed=2, std=3.0) if has_res else None
    g = None if gate is None else torch.sigmoid(rnd(*gate(T, H), dtype="fp32", seed=3)).to(TYPES[act])
    n1, s1 = spec(post, H, 10, wtype, **kw)
    n2, s2 = spec(pre, H, 20, wtype, **kw)
    h = torch.full((T, H), float("nan"), dtype=TYPES[res], device="cuda") if write_h else None
    y = torch.full((T, H), float("nan"), dtype=TYPES[act], device="cuda") if pre else None
    moe.moe_residual_norm(z, r, g, n1, alpha, h, n2, y, stream)
    rh, ry = S.residual_norm(f64(z), f64(r), f64(g), s1, alpha, s2)
    eh = 64 * 2.0 ** -24 * (abs(alpha) * terms(f64(z), s1) + np.abs(rh).max(axis=1, keepdims=True))
    if write_h:
        assert np.all(np.abs(f64(h) - rh) <= eh + half(h) * np.abs(rh))
    if pre:
        scale = S.norm(rh, **s2)[1] * (np.abs(s2["weight"] + s2.get("offset", 0.0)).max())
        ey = 64 * 2.0 ** -24 * terms(rh, s2) + 2 * eh * scale
        tiny = SMALLEST[y.dtype] / 2
        assert np.all(np.abs(f64(y) - ry) <= ey * (1 + half(y)) + half(y) * np.abs(ry) + tiny)
    return h, y


full, row, col = (lambda T, H: (T, H)), (lambda T, H: (T, 1)), (lambda T, H: (1, H))


@pytest.mark.parametrize("H", [1, 2, 7, 8, 63, 64, 255, 256, 1000, 2688, 2880, 4095, 4096, 4104, 8192, 16383, 16384])
def test_widths(H):
    run(5, H)
    run(3, H, act="fp32", res="fp32", post="layer", pre="layer", gate=full)


@pytest.mark.parametrize("act,res", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32"),
                                     ("fp32", "fp32")])
@pytest.mark.parametrize("gate", [None, full, row, col])
def test_types_and_gates(act, res, gate):
    for wtype in ("bf16", "fp16", "fp32"):
        run(9, 320, act, res, gate, wtype=wtype, alpha=0.3)
        run(9, 77, act, res, gate, "layer", "rms", wtype=wtype, alpha=-1.5, offset=1.0)


@pytest.mark.parametrize("post", [None, "rms", "layer"])
@pytest.mark.parametrize("pre", [None, "rms", "layer"])
def test_parts(post, pre):
    run(6, 512, post=post, pre=pre)
    run(6, 512, post=post, pre=pre, has_res=False)
    run(1, 2880, post=post, pre=pre, gate=row)
    if pre:
        run(6, 512, post=post, pre=pre, write_h=False)


@pytest.mark.parametrize("T", [1, 2, 151, 153, 1000, 5000])
def test_lengths(T):
    run(T, 2880, gate=col)


def test_large_mean():
    run(8, 2880, act="fp32", res="fp32", post="layer", pre="layer", mean=1000.0)


def test_only_the_pre_norm():
    r = rnd(7, 256, seed=5)
    y = torch.empty(7, 256, dtype=torch.bfloat16, device="cuda")
    n, s = spec("rms", 256, 3)
    moe.moe_residual_norm(None, r, None, None, 1.0, None, n, y)
    ref = S.norm(f64(r), **s)[0]
    assert np.all(np.abs(f64(y) - ref) <= half(y) * np.abs(ref) + 64 * 2.0 ** -24 * (1 + half(y)) * terms(f64(r), s))


def test_in_place_and_rows_apart():
    T, H = 33, 640
    want_h, want_y = run(T, H, "bf16", "fp32", row)
    z = torch.zeros(T, 3 * H, dtype=torch.bfloat16, device="cuda")
    zv = z[:, H:2 * H]
    zv.copy_(rnd(T, H, dtype="bf16", seed=1, std=2.0))
    r = rnd(T, H, dtype="fp32", seed=2, std=3.0)
    g = torch.sigmoid(rnd(T, 1, seed=3)).to(torch.bfloat16)
    moe.moe_residual_norm(zv, r, g, spec("rms", H, 10)[0], 1.0, r, spec("rms", H, 20)[0], zv)
    assert torch.equal(r, want_h) and torch.equal(zv, want_y)
    assert not z[:, :H].any() and not z[:, 2 * H:].any()


def test_all_zero_and_non_finite_rows():
    z = torch.zeros(3, 64, device="cuda")
    z[1, 5] = float("nan")
    r = torch.zeros(3, 64, device="cuda")
    h, y = torch.empty_like(r), torch.empty_like(r)
    n = moe.norm("rms")
    moe.moe_residual_norm(z, r, None, n, 1.0, h, n, y)
    assert not y[0].any() and torch.isnan(y[1]).all() and not y[2].any()


def test_captured_in_a_graph():
    T, H = 40, 2880
    z, r = rnd(T, H, dtype="bf16", seed=1), rnd(T, H, dtype="bf16", seed=2)
    h, y = torch.zeros_like(r), torch.zeros_like(z)
    n = moe.norm("rms", torch.ones(H, device="cuda"))
    n.tensors = None
    w = torch.ones(H, device="cuda")
    n = moe.norm("rms", w)
    moe.moe_residual_norm(z, r, None, n, 1.0, h, n, y)
    want = (h.clone(), y.clone())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        moe.moe_residual_norm(z, r, None, n, 1.0, h, n, y)
    h.zero_(), y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, want[0]) and torch.equal(y, want[1])


@pytest.mark.parametrize("H", [1, 5, 7, 9, 65, 1003, 2881, 4090, 8178, 8191])
def test_many_rows_off_the_grid(H):
    run(700, H, gate=row)
    run(700, H, "fp16", "fp32", full, "layer", "layer")
    run(700, H, "bf16", "fp32", col, None, "rms", alpha=-0.5)
    run(459, H, "fp32", "fp32", full, "rms", "layer", wtype="bf16")


@pytest.mark.parametrize("H,stride", [(640, 643), (641, 648), (100, 109), (3, 4), (8, 9), (13, 14)])
def test_many_rows_of_another_stride(H, stride):
    """Rows that lie `stride` apart: the same results as of rows that lie close, and nothing written between them."""
    T = 613
    want_h, want_y = run(T, H, "bf16", "fp32", row)

    def apart(dtype, rows=None):
        t = torch.full((T, stride), -7.0, dtype=dtype, device="cuda")
        if rows is not None:
            t[:, :H] = rows
        return t

    z = apart(torch.bfloat16, rnd(T, H, dtype="bf16", seed=1, std=2.0))
    r = apart(torch.float32, rnd(T, H, dtype="fp32", seed=2, std=3.0))
    g = torch.sigmoid(rnd(T, 1, seed=3)).to(torch.bfloat16)
    h, y = apart(torch.float32), apart(torch.bfloat16)
    moe.moe_residual_norm(z[:, :H], r[:, :H], g, spec("rms", H, 10)[0], 1.0, h[:, :H], spec("rms", H, 20)[0], y[:, :H])
    # the sums' order is another: 128 * 2^-24 of a row's largest value, and a step of the output's type
    top_h, top_y = want_h.abs().amax(1, keepdim=True), want_y.float().abs().amax(1, keepdim=True)
    assert ((h[:, :H] - want_h).abs() <= 128 * 2.0 ** -24 * (top_h + 8)).all()
    assert ((y[:, :H].float() - want_y.float()).abs() <= 2.0 ** -7 * want_y.float().abs() + 2.0 ** -16 * top_y).all()
    assert (h[:, H:] == -7).all() and (y[:, H:] == -7).all()
    # strides that differ
    r2, h2, y2 = apart(torch.float32)[:, :H], torch.empty(T, H, device="cuda"), apart(torch.bfloat16)
    r2.copy_(r[:, :H])
    moe.moe_residual_norm(z[:, :H], r2, g, spec("rms", H, 10)[0], 1.0, h2, spec("rms", H, 20)[0], y2[:, :H])
    assert ((h2 - want_h).abs() <= 128 * 2.0 ** -24 * (top_h + 8)).all() and (y2[:, H:] == -7).all()


def test_many_rows_in_place_off_the_grid():
    T, H = 1500, 331
    want_h, want_y = run(T, H, "bf16", "bf16", row)
    z, r = rnd(T, H, dtype="bf16", seed=1, std=2.0), rnd(T, H, dtype="bf16", seed=2, std=3.0)
    g = torch.sigmoid(rnd(T, 1, seed=3)).to(torch.bfloat16)
    moe.moe_residual_norm(z, r, g, spec("rms", H, 10)[0], 1.0, r, spec("rms", H, 20)[0], z)
    assert torch.equal(r, want_h) and torch.equal(z, want_y)


@pytest.mark.parametrize("H", [1000, 2048, 2880, 4096, 4104, 8192])
def test_many_rows_on_the_grid(H):
    """More than two rows an SM: every size of the walking kernel, with and without gates and biases."""
    T = 700
    run(T, H, gate=row)
    run(T, H, "bf16", "fp32", full, "layer", "layer")
    run(T, H, "fp16", "fp16", None, "rms", "layer", wtype="fp16", alpha=0.3)
    run(T, H, "fp16", "fp32", col, "layer", "rms")
    run(T, H, "fp32", "fp32", None, None, "rms", offset=1.0)
    run(T, H, "fp32", "fp32", full, "layer", None, alpha=-1.5)
    run(T, H, gate=row, has_res=False, write_h=False)


@pytest.mark.parametrize("H", [2880, 2881, 4104])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_only_the_pre_norm_of_many_rows(H, kind):
    r = rnd(700, H, seed=5)
    y = torch.empty(700, H, dtype=torch.bfloat16, device="cuda")
    n, s = spec(kind, H, 3)
    moe.moe_residual_norm(None, r, None, None, 1.0, None, n, y)
    ref = S.norm(f64(r), **s)[0]
    assert np.all(np.abs(f64(y) - ref) <= half(y) * np.abs(ref) + 64 * 2.0 ** -24 * (1 + half(y)) * terms(f64(r), s))
