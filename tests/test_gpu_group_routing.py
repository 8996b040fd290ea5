"""moe_route_grouped against the float64 oracle: the ids must be equal, ties included (sums of two scores that 64
bits do not tell apart excepted).

Weights: each exponential is off by at most 2 ulps (2^-22) and by its rounded argument (2^-24 of it), sums of up to
256 terms by at most 21 * 2^-24 (8 or 16 in a lane, five joins), two more roundings for the quotient and the factor:
|w - ref| <= ref * (2 * 2^-22 + span * 2^-23 + 24 * 2^-24) with the span of the logits that weigh."""
import numpy as np
import pytest
import torch

import bit_block_scaled_gb300 as moe
from gpu_helpers import built, ws_status
from oracle import group_routing as GR

pytestmark = pytest.mark.gpu
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def lib():
    return built()


def gpu(logits, bias, k, stream=None, **r):
    T = logits.shape[0]
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    ws = ws_status()
    moe.moe_route_grouped(logits, bias, k, moe.router(**r), ids, w, ws, stream)
    assert moe.moe_read_status(ws, stream) == 0
    return ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)


def below_64_bits(l, bias, score, n_group=1, topk_group=1, group_score="max", **_):
    """Whether the last kept and the first dropped group of a row differ, in more than 64 bits, but by less than a
    sum of two 64-bit scores resolves (2^-51 of it): either order is right."""
    if group_score != "top2" or topk_group == n_group or bias is None:
        return False
    l, b = l.astype(np.longdouble), bias.astype(np.longdouble)
    assert np.finfo(np.longdouble).nmant > 60
    s = np.exp(l - l.max()) if score == "softmax" else 1 / (1 + np.exp(-l))
    c = (s / s.sum() if score == "softmax" else s) + b
    g = np.sort(np.sort(c.reshape(n_group, -1), axis=1)[:, -2:].sum(axis=1))[::-1]
    gap = g[topk_group - 1] - g[topk_group]
    return 0 < gap <= abs(g[topk_group]) * 2.0 ** -51


def check(logits, bias, k, **r):
    ids, w = gpu(logits, bias, k, **r)
    l = logits.float().cpu().numpy()
    rid, rw = GR.route_grouped(l, None if bias is None else bias.cpu().numpy(), k, **r)
    for t in np.flatnonzero((ids != rid).any(axis=1)):
        assert below_64_bits(l[t], None if bias is None else bias.cpu().numpy(), **r), t
    rw = np.where((ids == rid).all(axis=1, keepdims=True), rw, w)
    f = l[np.isfinite(l)]
    span = float(np.ptp(f)) if f.size else 0.0
    tol = 2 * 2.0 ** -22 + span * 2.0 ** -23 + 24 * 2.0 ** -24
    assert np.all(np.abs(w - rw) <= np.abs(rw) * tol + 2.0 ** -126)  # subnormal weights keep an absolute error
    return ids, w


def draw(T, E, dtype="fp32", seed=0, std=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * std).to(TYPES[dtype]).cuda()


def bias_of(E, seed=1, std=0.1):
    return (torch.randn(E, generator=torch.Generator().manual_seed(seed)) * std).cuda()


@pytest.mark.parametrize("E,k,n_group,topk_group", [
    (1, 1, 1, 1), (2, 1, 2, 1), (8, 2, 1, 1), (33, 4, 1, 1), (64, 8, 8, 3), (96, 6, 4, 2), (128, 6, 1, 1),
    (129, 5, 3, 2), (160, 8, 5, 2), (252, 8, 9, 4), (255, 7, 17, 5), (256, 8, 8, 4), (256, 8, 32, 1), (256, 1, 2, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_shapes(E, k, n_group, topk_group, score, with_bias):
    for gscore in ("max", "top2"):
        if gscore == "top2" and E // n_group < 2:
            continue
        for i, dtype in enumerate(("fp32", "bf16", "fp16")):
            check(draw(37, E, dtype, seed=E + i), bias_of(E) if with_bias else None, k, score=score, n_group=n_group,
                  topk_group=topk_group, group_score=gscore, renormalize=i != 1, scale=(1.0, 2.5, 0.0)[i])


@pytest.mark.parametrize("T", [1, 2, 3, 5, 1000, 8193])
def test_lengths(T):
    check(draw(T, 256, seed=T), bias_of(256), 8, score="sigmoid", n_group=8, topk_group=4, group_score="top2", scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("gscore", ["max", "top2"])
def test_exact_and_near_ties(score, gscore):
    """Few distinct logits: most choices are exact ties. Then logits one ulp apart, whose fp32 scores with the bias
    round to the same or to the wrong order: the choice has to follow the real scores."""
    rng = np.random.default_rng(3)
    r = dict(score=score, n_group=8, topk_group=3, group_score=gscore)
    l = torch.from_numpy(rng.integers(-2, 3, size=(200, 64)).astype(np.float32)).cuda()
    for bias in (None, torch.zeros(64, device="cuda"),
                 torch.from_numpy(rng.integers(0, 2, 64).astype(np.float32)).cuda()):
        check(l, bias, 6, **r)
    base = rng.normal(size=(300, 1)).astype(np.float32)
    steps = rng.integers(0, 40, size=(300, 64))
    near = (base.view(np.int32) + steps.astype(np.int32)).view(np.float32)
    for bias in (torch.zeros(64, device="cuda"), torch.full((64,), 1000.0, device="cuda")):
        ids, _ = check(torch.from_numpy(near).cuda(), bias, 6, **r)
    assert not np.array_equal(ids[:, 0], np.zeros(300))  # not all decided by the index


def test_minus_zero_ties_with_zero():
    l = torch.tensor([[-0.0, 0.0, -0.0, -1.0]], device="cuda")
    ids, _ = check(l, None, 3)
    assert ids.tolist() == [[0, 1, 2]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_non_finite_rows(score, with_bias, renorm):
    nan, inf = float("nan"), float("inf")
    rng = np.random.default_rng(4)
    rows = [np.full(32, nan), np.full(32, -inf), np.full(32, inf), np.zeros(32)]
    for v, n in ((nan, 20), (inf, 2), (-inf, 30), (-inf, 4), (nan, 31)):
        r = rng.integers(-2, 3, 32).astype(np.float64)
        r[rng.choice(32, n, replace=False)] = v
        rows.append(r)
    l = torch.from_numpy(np.stack(rows).astype(np.float32)).cuda()
    bias = bias_of(32) if with_bias else None
    check(l, bias, 4, score=score, renormalize=renorm)
    check(l, bias, 4, score=score, renormalize=renorm, n_group=4, topk_group=2, group_score="max")
    check(l, bias, 4, score=score, renormalize=renorm, n_group=4, topk_group=2, group_score="top2")


def test_far_negative_sigmoids_keep_their_ratios():
    l = torch.linspace(-300, -290, 16, device="cuda").repeat(3, 1)
    _, w = check(l, None, 4, score="sigmoid")
    assert np.allclose(w.sum(axis=1), 1.0) and w[0, 0] > w[0, 3]


def test_rows_apart_and_another_stream():
    wide = draw(50, 200, "bf16", seed=9)
    l = wide[:, 64:64 + 96]
    ids, w = gpu(l, None, 4)
    rid, _ = GR.route_grouped(l.float().cpu().numpy(), None, 4)
    assert np.array_equal(ids, rid)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ids2, w2 = gpu(l, None, 4)
    s.synchronize()
    assert np.array_equal(ids, ids2) and np.array_equal(w, w2)


def test_agrees_with_the_plain_router():
    l = draw(500, 128, seed=11)
    ids = torch.empty(500, 6, dtype=torch.int32, device="cuda")
    w = torch.empty(500, 6, device="cuda")
    moe.moe_route_topk(l, None, 6, moe.ROUTE["topk_softmax"], ids, w, ws_status())
    gid, gw = gpu(l, None, 6)
    assert np.array_equal(ids.cpu().numpy(), gid)
    np.testing.assert_allclose(w.cpu().numpy(), gw, rtol=2e-6)


@pytest.mark.parametrize("std,bias_std", [(2.0, 0.003), (2.0, 0.1), (0.01, 1e-6), (30.0, 0.01)])
def test_softmax_with_a_bias_near_ties(std, bias_std):
    """Softmax scores of many experts lie close together: a gap of the order of the bias's and of fp32's rounding
    decides in some rows of every batch. With wide logits most scores vanish beside the bias."""
    l = draw(3000, 256, seed=5, std=std)
    l[::7, 40:90] = float("-inf")
    b = bias_of(256, std=bias_std)
    b[8:16] = b[:8]  # the bias alone ties
    for r in (dict(), dict(n_group=8, topk_group=4, group_score="top2"), dict(n_group=8, topk_group=4)):
        check(l, b, 8, score="softmax", **r)
    check(l, None, 8, score="softmax", n_group=16, topk_group=5, group_score="top2", renormalize=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n_group,topk_group", [(2, 1), (8, 3)])
@pytest.mark.parametrize("size,spread", [(64.0, 1e-2), (256.0, 1e-2), (256.0, 1e-4), (1e6, 1e-4), (1e6, 4e-8), (0.0, 1e-2)])
def test_biases_of_opposite_sign_in_a_group(score, n_group, topk_group, size, spread):
    """A group's two best scores carry the rounding of their own size, which their sum may have lost: biases +B and -B
    in a group, larger and smaller B side by side. Groups of two, all of whose experts are chosen with them; the groups
    of a row are those of the sums in long double, unless the last kept and the first dropped are closer than 64-bit
    scores of that size resolve (two roundings of each of the two scores of the two groups)."""
    T, E, k = 20000, 2 * n_group, 2 * topk_group
    b = np.zeros((n_group, 2), np.float32)
    b[:, 0] = size * (1.0 if n_group == 2 else np.resize([1.0, 0.5, 1.0, 0.0], n_group))
    b[:, 1] = -b[:, 0]
    g = torch.Generator().manual_seed(17)
    l = torch.randn(T, E, generator=g) * spread
    ids, _ = gpu(l.cuda(), torch.from_numpy(b.reshape(-1)).cuda(), k, score=score, n_group=n_group,
                 topk_group=topk_group, group_score="top2")
    x = l.numpy().astype(np.longdouble)
    assert np.finfo(np.longdouble).nmant > 60
    s = np.exp(x) / np.exp(x).sum(axis=1, keepdims=True) if score == "softmax" else 1 / (1 + np.exp(-x))
    sums = (s.reshape(T, n_group, 2) + b).sum(axis=2)
    order = np.argsort(-sums, axis=1, kind="stable")
    ranked = np.take_along_axis(sums, order, axis=1)
    open_ = ranked[:, topk_group - 1] - ranked[:, topk_group] <= 8 * 2.0 ** -53 * (1 + size)
    want = np.sort(order[:, :topk_group], axis=1)
    got = np.sort(ids // 2, axis=1)[:, ::2]
    wrong = (got != want).any(axis=1) & ~open_
    assert open_.mean() < 0.6 and not wrong.any(), (int(wrong.sum()), int(open_.sum()))


def test_sums_that_lose_what_pairs_of_floats_hold():
    """Biases of +-1e6 next to scores that differ by a few steps of fp32 (some 2e-9): pairs of floats are off by that
    much there, so the row has to go on to 64 bits."""
    T, size = 600000, 1e6
    rng = np.random.default_rng(5)
    l = np.repeat(rng.uniform(-0.1, 0.1, size=(T, 1, 2)).astype(np.float32), 2, axis=1)
    l = (l.view(np.int32) + rng.integers(0, 4, size=l.shape).astype(np.int32)).view(np.float32)
    b = np.array([size, -size] * 2, np.float32)
    ids, _ = gpu(torch.from_numpy(l.reshape(T, 4)).cuda(), torch.from_numpy(b).cuda(), 2, score="sigmoid", n_group=2,
                 topk_group=1, group_score="top2")
    gap = (1 / (1 + np.exp(-l.astype(np.longdouble)))).sum(axis=2) @ np.array([1.0, -1.0])
    open_ = np.abs(gap) <= 8 * 2.0 ** -53 * (1 + size)
    wrong = (ids[:, 0] // 2 != (gap < 0)) & ~open_
    assert open_.mean() < 0.5 and not wrong.any(), (int(wrong.sum()), int(open_.sum()))


@pytest.mark.parametrize("top", [5.0, 0.0, -5.0, -20.0, -29.0, -31.0, -60.0])
@pytest.mark.parametrize("renorm", [False, True])
def test_sigmoids_far_below_the_largest_chosen(top, renorm):
    """Ratios are kept where a sigmoid by itself is subnormal (logits below -87) and the largest is not: renormalised
    weights have the error of any other, down to fp32's normal range."""
    g = torch.Generator().manual_seed(21)
    l = top - 83 * torch.rand(400, 8, generator=g)
    l[:, 3] = top
    l[::2, 5] = -95.0 - torch.rand(200, generator=g)
    check(l.cuda(), None, 8, score="sigmoid", renormalize=renorm)
    check(l.cuda(), bias_of(8, std=100.0), 4, score="sigmoid", renormalize=renorm, n_group=4, topk_group=3)
