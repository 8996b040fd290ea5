"""moe_rope and moe_rope_kv_write against float64: layouts, parts of a head, far positions, types, strides, in place."""
import numpy as np
import pytest
import torch

import bit_block_scaled_gb300 as moe
from gpu_helpers import built, ws_status
from oracle import kvcache as KV
from oracle import rope as R

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def lib():
    return built()


def f64(t):
    return t.double().cpu().numpy()


def make(T, heads, D, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, heads, D, generator=g).to(dtype).cuda()


def positions(T, far=100000, seed=0):
    g = torch.Generator().manual_seed(seed + 77)
    return torch.randint(-far, far, (T,), generator=g, dtype=torch.int32).cuda()


def reference(x, pos, rope, layout):
    turns = rope.table.cpu().numpy().view(np.uint64)
    return R.rotate(f64(x), R.angles(pos.cpu().numpy(), turns), layout, rope.amplitude)


def close(got, x, ref, dtype, rot):
    """Half a step of the output; cosine and sine off by 2^-22 at most (two last bits of fp32 and the angle's own
    2^-26 of a turn's eighth), the two products and their sum by 2^-24 each, of the pair's magnitudes."""
    big = np.abs(f64(x)).max(axis=-1, keepdims=True)
    tol = torch.finfo(dtype).eps / 2 * np.abs(ref) + 4 * 2.0 ** -22 * big * 2
    assert (np.abs(f64(got) - ref) <= tol).all()
    assert torch.equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,hq,hk,D,rot", [(1, 64, 8, 64, 64), (3, 1, 1, 128, 128), (17, 5, 3, 128, 64), (300, 8, 8, 256, 256),
                                          (700, 40, 8, 64, 32), (5, 7, 2, 80, 80), (9, 3, 1, 48, 16), (33, 4, 2, 64, 20),
                                          (6, 2, 3, 50, 6), (2, 3, 1, 3, 2), (40, 2, 1, 256, 254), (1, 33, 0, 128, 96), (7, 3, 2, 72, 64),
                                          (31, 5, 1, 72, 70), (700, 6, 2, 128, 102), (4, 9, 9, 8, 4), (400, 3, 2, 248, 30)])
def test_rope(layout, dtype, T, hq, hk, D, rot):
    t = TYPES[dtype]
    r = moe.rope(rot, layout, 10000.0)
    q, k, pos = make(T, hq, D, t), make(T, hk, D, t, 1), positions(T)
    qo, ko = torch.full_like(q, 7), torch.full_like(k, 7)
    moe.moe_rope(r, pos, q, qo, *((k, ko) if hk else ()))
    close(qo, q, reference(q, pos, r, layout), t, rot)
    if hk:
        close(ko, k, reference(k, pos, r, layout), t, rot)


@pytest.mark.parametrize("kw", [dict(scaling="yarn", factor=32.0, base=150000.0, truncate=False),
                                dict(scaling="llama3", factor=8.0, base=500000.0), dict(scaling="ntk", factor=4.0),
                                dict(scaling="linear", factor=4.0), dict(amplitude=0.5)])
def test_scalings_at_far_positions(kw):
    """Against the definition in float64, whose own angle at 2^31 is good to 2^31 2^-53."""
    r = moe.rope(64, "half", **kw)
    pos = torch.tensor([0, 1, -1, 4095, 131072, 10 ** 6, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32).cuda()
    q = make(len(pos), 2, 64, torch.float32)
    out = torch.empty_like(q)
    moe.moe_rope(r, pos, q, out)
    f, amp = R.frequencies(64, **{k: v for k, v in kw.items() if k != "amplitude"})
    ref = R.rotate(f64(q), pos.cpu().numpy().astype(np.float64)[:, None] * f, "half", kw.get("amplitude", amp))
    big = np.abs(f64(q)).max(axis=-1, keepdims=True)
    assert (np.abs(f64(out) - ref) <= 2.0 ** -24 * np.abs(ref) + (8 * 2.0 ** -22 + 2.0 ** -20) * big).all()


def test_frequencies_of_the_callers():
    f = np.array([0.5, 7.0, 1e-4, 0.0])
    r = moe.rope(8, "interleaved", frequencies=f, amplitude=2.0)
    q, pos = make(5, 2, 8, torch.float32), torch.arange(5, dtype=torch.int32).cuda()
    out = torch.empty_like(q)
    moe.moe_rope(r, pos, q, out)
    ref = R.rotate(f64(q), np.outer(np.arange(5), f), "interleaved", 2.0)
    np.testing.assert_allclose(f64(out), ref, atol=4e-6)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 40), (64, 16), (256, 250), (128, 34), (72, 54), (50, 50)])
def test_in_place_and_strided(layout, D, rot):
    """Parts of a projection's output, rotated where they lie; what is beside them stays."""
    T, hq, hk = 700, 6, 2
    r, pos = moe.rope(rot, layout), positions(T)
    qkv = make(T, hq + 2 * hk, D, torch.bfloat16)
    before = qkv.clone()
    q, k, v = qkv.split((hq, hk, hk), dim=1)
    a, b = torch.empty(T, hq, D, dtype=torch.bfloat16, device="cuda"), torch.empty(T, hk, D, dtype=torch.bfloat16, device="cuda")
    moe.moe_rope(r, pos, q, a, k, b)
    moe.moe_rope(r, pos, q, q, k, k)
    assert torch.equal(q, a) and torch.equal(k, b) and torch.equal(v, before[:, hq + hk:])
    heads_first = make(hq, T, D, torch.bfloat16)  # [heads, T, D]
    x = heads_first.transpose(0, 1)
    y = torch.zeros(T, hq, D + 3, dtype=torch.bfloat16, device="cuda")  # rows off the 16-byte grid
    moe.moe_rope(r, pos, x, y[..., :D])
    close(y[..., :D], x, reference(x, pos, r, layout), torch.bfloat16, rot)
    assert (y[..., D:] == 0).all()
    one = make(1, 1, D, torch.bfloat16).expand(T, hq, D)  # one head for all
    z = torch.empty(T, hq, D, dtype=torch.bfloat16, device="cuda")
    moe.moe_rope(r, pos, one, z)
    close(z, one, reference(one, pos, r, layout), torch.bfloat16, rot)


def test_back_again_and_relative():
    """Negative positions undo a rotation, and products of rotated vectors depend on the distance alone."""
    r = moe.rope(128, "half", 500000.0)
    q, k = make(1, 1, 128, torch.float32), make(1, 1, 128, torch.float32, 1)

    def at(x, p):
        y = torch.empty_like(x)
        moe.moe_rope(r, torch.tensor([p], dtype=torch.int32, device="cuda"), x, y)
        return y
    for p in (1, 1234567, 2 ** 31 - 1):
        assert (at(at(q, p), -p) - q).abs().max() < 2e-6
    dots = [(at(q, p + 100) * at(k, p)).sum().item() for p in (0, 1000, 10 ** 6, 10 ** 9)]
    assert max(dots) - min(dots) < 1e-4


def cache_of(fmt, pages, page, heads, D):
    data = torch.zeros(pages, heads, page // 16, moe.moe_kv_record_bytes(fmt, D), dtype=torch.uint8, device="cuda")
    return data, moe.kv_cache(data, fmt, D)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("fmt", ["bf16", "fp16", "fp8", "nvfp4"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,hq,hk,D,rot,page", [(1, 64, 8, 64, 64, 16), (70, 3, 1, 64, 64, 32), (45, 4, 2, 128, 64, 16),
                                               (333, 6, 3, 256, 256, 48), (19, 2, 5, 64, 20, 16), (150, 2, 2, 128, 102, 16)])
def test_write(layout, fmt, dtype, T, hq, hk, D, rot, page):
    t = TYPES[dtype]
    r, pos = moe.rope(rot, layout, 150000.0), positions(T)
    qkv = make(T, hq + 2 * hk, D, t, T)
    q, k, v = qkv.split((hq, hk, hk), dim=1)
    pages = T // page + 3
    data, c = cache_of(fmt, pages, page, hk, D)
    plain, cp = cache_of(fmt, pages, page, hk, D)
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(T))[:T].to(torch.int32).cuda()
    slots[T // 2] = -1
    out, ws = torch.full((T, hq, D), 7.0, dtype=t, device="cuda"), ws_status()
    moe.moe_rope_kv_write(r, pos, q, out, k, v, slots, c, ws)
    want = torch.empty_like(out)
    moe.moe_rope(r, pos, q, want)
    assert torch.equal(out, want)  # as without the cache
    # the same bytes as a write of the rotated keys in fp32; values and what is not written too
    kr = torch.empty(T, hk, D, device="cuda")
    moe.moe_rope(r, pos, k.float(), kr)
    moe.moe_kv_write(kr, v.float(), slots, cp, ws)
    assert torch.equal(data, plain)
    # and no query
    again, ca = cache_of(fmt, pages, page, hk, D)
    moe.moe_rope_kv_write(r, pos, None, None, k, v, slots, ca, ws)
    assert torch.equal(again, data) and moe.moe_read_status(ws) == 0


def test_write_past_the_cache():
    data, c = cache_of("fp8", 2, 16, 2, 64)
    r, ws = moe.rope(64), ws_status()
    k = make(3, 2, 64, torch.bfloat16)
    moe.moe_rope_kv_write(r, positions(3), None, None, k, k, torch.tensor([32, -5, 3], dtype=torch.int32, device="cuda"), c, ws)
    assert moe.moe_read_status(ws) == 5
    keys, _ = KV.values(data.cpu().numpy(), "fp8", 64)
    assert np.count_nonzero(np.abs(keys).sum(axis=-1)) == 2  # the third token's two heads


def test_keys_without_numbers():
    data, c = cache_of("nvfp4", 1, 16, 1, 64)
    r, ws = moe.rope(64), ws_status()
    k = make(2, 1, 64, torch.bfloat16)
    v = k.clone()
    k[0, 0, 3] = float("nan")
    ko, vo = torch.empty(2, 1, 64, device="cuda"), torch.empty(2, 1, 64, device="cuda")
    s = torch.arange(2, dtype=torch.int32, device="cuda")
    moe.moe_rope_kv_write(r, positions(2), None, None, k, v, s, c, ws)
    moe.moe_kv_read(c, s, ko, vo, ws)
    assert torch.isnan(ko[0]).all() and not torch.isnan(ko[1]).any() and not torch.isnan(vo).any()
