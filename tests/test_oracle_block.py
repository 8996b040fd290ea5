"""CPU pins of the oracles of the calls around the layer: closed forms, brute force, round trips."""
import itertools

import numpy as np
import pytest

from oracle import group_routing as GR
from oracle import kvcache as KV
from oracle import routing as R
from oracle import seam as S


def test_one_group_is_the_plain_router():
    rng = np.random.default_rng(0)
    l = rng.normal(size=(50, 32)).astype(np.float32)
    ids, w = GR.route_grouped(l, None, 4, "softmax")
    rid, rw = R.topk_softmax(l, 4)
    assert np.array_equal(ids, rid)
    np.testing.assert_allclose(w, rw, rtol=1e-6)
    b = rng.normal(size=32).astype(np.float32)
    ids, w = GR.route_grouped(l, b, 4, "sigmoid")
    rid, rw = R.sigmoid_bias_topk(l, b, 4)
    same = (ids == rid).all(axis=1)
    assert same.mean() > 0.9
    np.testing.assert_allclose(w[same], rw[same], rtol=1e-5)


@pytest.mark.parametrize("gscore", ["max", "top2"])
def test_groups_by_brute_force(gscore):
    rng = np.random.default_rng(1)
    l = rng.integers(-3, 4, size=(40, 12)).astype(np.float32)
    bias = rng.integers(0, 2, size=12).astype(np.float32)
    ids, _ = GR.route_grouped(l, bias, 3, "sigmoid", 4, 2, gscore)
    c = 1 / (1 + np.exp(-l.astype(np.float64))) + bias
    for t in range(40):
        g = [sorted(c[t, 3 * i:3 * i + 3])[::-1] for i in range(4)]
        v = [x[0] if gscore == "max" else x[0] + x[1] for x in g]
        keep = min(itertools.permutations(range(4), 2), key=lambda p: [(-v[i], i) for i in p])
        cand = [e for e in range(12) if e // 3 in keep]
        assert list(ids[t]) == sorted(cand, key=lambda e: (-c[t, e], e))[:3]


def test_router_weights_without_renormalising():
    l = np.array([[0.0, 0.0, 0.0, 0.0]], np.float32)
    ids, w = GR.route_grouped(l, None, 2, "softmax", renormalize=False, scale=2.0)
    assert ids.tolist() == [[0, 1]] and np.allclose(w, 0.5)
    _, w = GR.route_grouped(np.full((1, 4), -np.inf, np.float32), None, 2, "softmax")
    assert np.allclose(w, 0.5)
    _, w = GR.route_grouped(np.array([[-900.0, -901.0]], np.float32), None, 2, "sigmoid")
    assert np.allclose(w, [[1 / (1 + np.e ** -1), np.e ** -1 / (1 + np.e ** -1)]])


def test_seam_closed_forms():
    x = np.array([[3.0, 4.0]])
    y, _ = S.norm(x, "rms", eps=0.0)
    assert np.allclose(y, x / np.sqrt(12.5))
    y, _ = S.norm(x, "layer", eps=0.0)
    assert np.allclose(y, [[-1.0, 1.0]])
    h, y = S.residual_norm(x, np.ones((1, 2)), 0.5, None, 2.0, dict(kind="rms", eps=0.0))
    assert np.allclose(h, [[4.0, 5.0]]) and np.allclose(y, h / np.sqrt(20.5))
    h, y = S.residual_norm(None, x, None, None, 1.0, None)
    assert np.array_equal(h, x) and y is None


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
def test_quantiser(fmt):
    rng = np.random.default_rng(2)
    x = rng.normal(size=(200, 64)) * np.exp(rng.normal(size=(200, 1)) * 5)
    x[3] = 0.0
    c, s, e = KV.quantise(x, fmt)
    v = KV.decode(c, s, e, fmt)
    amax = np.abs(x).max(axis=1, keepdims=True)
    # E4M3 is off by at most 2^-4 of a value; E2M1 by half its widest step, 1 of 6, of the largest of 16 and
    # the block scale by 2^-4
    tol = np.abs(x) * 2 ** -4 + amax * 2 ** -16 if fmt == "fp8" else \
        np.repeat(np.abs(x).reshape(200, 4, 16).max(axis=2), 16, axis=1) * (1 / 6 + 2 ** -4) + amax * 2 ** -10
    assert np.all(np.abs(v - x) <= tol)
    top = 448.0 if fmt == "fp8" else 2688.0
    r = 2.0 ** (e.astype(float) - 127)
    live = amax[:, 0] > 0
    assert np.all(amax[live, 0] / r[live] <= top) and np.all(amax[live, 0] / r[live] > top / 2)
    assert e[3] == 0 and np.all(v[3] == 0)
    x[5, 7] = np.inf
    c, s, e = KV.quantise(x, fmt)
    assert e[5] == 255 and np.all(c[5] == 0) and np.isnan(KV.decode(c, s, e, fmt)[5]).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_places_are_a_permutation_within_lines(fmt, D):
    p = KV.place(fmt, D)
    assert sorted(p.reshape(-1).tolist()) == list(range(16 * KV.row_bytes(fmt, D)))
    assert np.all(p // 128 == (np.arange(16)[:, None] * KV.row_bytes(fmt, D) + np.arange(KV.row_bytes(fmt, D))) // 128)


def test_attention_closed_forms():
    keys, vals = np.zeros((1, 1, 16, 2)), np.zeros((1, 1, 16, 2))
    vals[0, 0, :3, 0] = [1.0, 2.0, 6.0]
    q = np.zeros((1, 1, 2))
    out, lse, _, _, _ = KV.attend(q, keys, vals, np.array([[0]]), [3], 1.0)
    assert np.allclose(out[0, 0], [3.0, 0.0]) and np.allclose(lse, np.log(3))
    out, lse, _, _, _ = KV.attend(q, keys, vals, np.array([[0]]), [3], 1.0, window=1, sinks=np.array([0.0]))
    assert np.allclose(out[0, 0], [3.0, 0.0]) and np.allclose(lse, np.log(2))
    out, lse, _, _, _ = KV.attend(q, keys, vals, np.array([[0]]), [0], 1.0)
    assert np.all(out == 0) and np.all(lse == -np.inf)
    out, lse, _, _, _ = KV.attend(q, keys, vals, np.array([[7]]), [3], 1.0)
    assert np.all(out == 0) and np.all(lse == -np.inf)
