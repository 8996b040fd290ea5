"""moe_kv_write and moe_kv_read against the float64 oracle, byte by byte: row scales are powers of two, so codes,
block scales and exponents are those of real arithmetic for 16-bit inputs, and what is read back is exact up to its
rounding to the output's type."""
import numpy as np
import pytest
import torch

import bit_block_scaled_gb300 as moe
from gpu_helpers import built, ws_status
from oracle import kvcache as KV

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def lib():
    return built()


def tokens(T, H, D, dtype, seed=0):
    """Rows of very different sizes, all-zero ones and zeros of both signs among them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, D, generator=g) * torch.exp(2 * torch.randn(T, H, 1, generator=g))
    x[:, :, 3::17] = 0.0
    x[:, :, 5::19] = -0.0
    x[::5, 0] = 0.0
    return x.to(TYPES[dtype]).cuda()


def new_cache(fmt, D, H, pages, page, fill=0):
    data = torch.full((pages, H, page // 16, KV.record_bytes(fmt, D)), fill, dtype=torch.uint8, device="cuda")
    return data, moe.kv_cache(data, fmt, D)


def stored(rec, i, part, fmt, D):
    codes, sc, ex = KV.unpack_record(rec, fmt, D)[part]
    return codes[i], None if sc is None else sc[i], None if ex is None else ex[i]


def check_written(data, slots, k, v, fmt, page):
    d = data.cpu().numpy()
    for part, x in ((0, k), (1, v)):
        x64 = x.double().cpu().numpy()
        if fmt in ("fp8", "nvfp4"):
            c, s, e = KV.quantise(x64, fmt)
        else:
            c = x.to(TYPES[fmt]).contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
            s = e = None
        for t, slot in enumerate(slots.tolist()):
            if slot < 0:
                continue
            for h in range(x.shape[1]):
                rec = d[slot // page, h, slot % page // 16]
                gc, gs, ge = stored(rec, slot % 16, part, fmt, x.shape[2])
                assert np.array_equal(gc, c[t, h]), (t, h, part)
                if s is not None:
                    assert np.array_equal(gs, s[t, h])
                if e is not None:
                    assert ge == e[t, h]


@pytest.mark.parametrize("fmt", ["bf16", "fp16", "fp8", "nvfp4"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_written_bytes_and_read_back(fmt, D):
    for act, page, H, T in (("bf16", 16, 3, 37), ("fp16", 48, 1, 5), ("fp32", 128, 2, 20)):
        if act == "fp32" and fmt in ("fp8", "nvfp4"):
            k, v = (tokens(T, H, D, "bf16", s).float() for s in (1, 2))
        else:
            k, v = tokens(T, H, D, act, 1), tokens(T, H, D, act, 2)
        if fmt == "fp16" and act != "fp16":
            k, v = k.clamp(-60000, 60000), v.clamp(-60000, 60000)
        pages = T // page + 3
        data, c = new_cache(fmt, D, H, pages, page, fill=0xA5)
        before = data.clone()
        slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(3))[:T].to(torch.int32)
        slots[T // 2] = -1
        ws = ws_status()
        moe.moe_kv_write(k, v, slots.cuda(), c, ws)
        assert moe.moe_read_status(ws) == 0
        check_written(data, slots, k, v, fmt, page)
        # what belongs to other slots is as it was
        back = data.clone()
        moe.moe_kv_write(k, v, slots.cuda(), moe.kv_cache(before, fmt, D), ws)
        assert torch.equal(before, back)
        out = [torch.full((T, H, D), float("nan"), dtype=TYPES["bf16" if act == "fp32" else act], device="cuda")
               for _ in range(2)]
        moe.moe_kv_read(c, slots.cuda(), out[0], out[1], ws)
        for x, o in ((k, out[0]), (v, out[1])):
            x64 = x.double().cpu().numpy()
            ref = KV.decode(*KV.quantise(x64, fmt), fmt) if fmt in ("fp8", "nvfp4") else x.to(TYPES[fmt]).double().cpu().numpy()
            ref = torch.from_numpy(ref).to(o.dtype)
            ref[T // 2] = 0
            assert torch.equal(o.cpu(), ref)


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
def test_every_value_of_a_row_scale(fmt):
    """Rows whose largest value is each power of two, and just above and below the borders of the row scale."""
    D = 64
    rows = []
    for e in range(-133, 128):
        for m in (1.0, 1.75, 1.7578125, 1.3125, 1.3203125, 1.9921875):
            rows.append(m * 2.0 ** e)
    top = torch.tensor(rows, dtype=torch.float64).to(torch.bfloat16)
    x = (top[:, None, None].double() * torch.linspace(-1, 1, D, dtype=torch.float64)).to(torch.bfloat16)
    x[:, :, -1] = top[:, None]
    T = x.shape[0]
    x = x.cuda()
    data, c = new_cache(fmt, D, 1, T // 16 + 1, 16)
    slots = torch.arange(T, dtype=torch.int32)
    moe.moe_kv_write(x, -x, slots.cuda(), c, ws_status())
    check_written(data, slots, x, -x, fmt, 16)


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
def test_rows_with_nan_or_infinity(fmt):
    k = tokens(4, 2, 64, "bf16")
    v = k.clone()
    k[0, 0, 3], k[1, 1, 63], v[2, 0, 0] = float("nan"), float("inf"), -float("inf")
    data, c = new_cache(fmt, 64, 2, 1, 16)
    slots = torch.arange(4, dtype=torch.int32)
    ws = ws_status()
    moe.moe_kv_write(k, v, slots.cuda(), c, ws)
    check_written(data, slots, k, v, fmt, 16)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    moe.moe_kv_read(c, slots.cuda(), ko, vo, ws)
    assert torch.isnan(ko[0, 0]).all() and torch.isnan(ko[1, 1]).all() and torch.isnan(vo[2, 0]).all()
    assert torch.isfinite(ko[2:]).all() and torch.isfinite(vo[0]).all() and torch.isfinite(ko[0, 1]).all()


def test_slots_past_the_cache():
    k = tokens(3, 1, 64, "bf16")
    data, c = new_cache("bf16", 64, 1, 2, 16)
    slots = torch.tensor([5, 32, -3], dtype=torch.int32, device="cuda")
    ws = ws_status()
    moe.moe_kv_write(k, k, slots, c, ws)
    assert moe.moe_read_status(ws) == 5
    moe.moe_clear_status(ws)
    ko = torch.full_like(k, float("nan"))
    moe.moe_kv_read(c, slots, ko, None, ws)
    assert moe.moe_read_status(ws) == 5
    assert torch.equal(ko[0], k[0]) and not ko[1:].any()


def test_strided_inputs_and_outputs_and_another_stream():
    T, H, D = 19, 4, 128
    qkv = tokens(T, 3 * H, D, "bf16", 7)
    k, v = qkv[:, H:2 * H], qkv[:, 2 * H:]
    kt = k.transpose(0, 1).contiguous().transpose(0, 1)  # heads outermost
    slots = torch.arange(T, dtype=torch.int32, device="cuda") * 2
    data, c = new_cache("nvfp4", D, H, 4, 16)
    moe.moe_kv_write(k, v, slots, c, ws_status())
    data2, c2 = new_cache("nvfp4", D, H, 4, 16)
    out = torch.zeros(H, T, 2, D, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ws = ws_status()
        moe.moe_kv_write(kt, v, slots, c2, ws)
        moe.moe_kv_read(c2, slots, out[:, :, 0].transpose(0, 1), out[:, :, 1].transpose(0, 1), ws)
    s.synchronize()
    assert torch.equal(data, data2)
    ko, vo = torch.empty_like(kt), torch.empty_like(v)
    moe.moe_kv_read(c, slots, ko, vo, ws_status())
    assert torch.equal(out[:, :, 0].transpose(0, 1), ko) and torch.equal(out[:, :, 1].transpose(0, 1), vo)


def test_a_cache_past_four_gigabytes():
    D, H, page, pages = 128, 8, 128, 20000
    data, c = new_cache("bf16", D, H, pages, page)
    assert data.numel() > 1 << 32
    k, v = tokens(4, H, D, "bf16", 1), tokens(4, H, D, "bf16", 2)
    slots = torch.tensor([0, pages * page - 1, pages * page // 2 + 7, 17], dtype=torch.int32, device="cuda")
    ws = ws_status()
    moe.moe_kv_write(k, v, slots, c, ws)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    moe.moe_kv_read(c, slots, ko, vo, ws)
    assert torch.equal(ko, k) and torch.equal(vo, v) and moe.moe_read_status(ws) == 0
    assert torch.equal(data[-1, -1, -1].cpu(), data[-1, -1, -1].cpu())
    rec = data[-1, H - 1, page // 16 - 1].cpu().numpy()
    assert np.array_equal(stored(rec, 15, 0, "bf16", D)[0], k[1, H - 1].view(torch.int16).cpu().numpy().view(np.uint16))


def bytes_of(slots, heads, fmt, D, page, shape):
    """Which bytes of a cache of that shape belong to the slots."""
    own = np.zeros(shape, dtype=bool)
    R, at = KV.row_bytes(fmt, D), KV.place(fmt, D)
    for slot in slots:
        i = slot % 16
        for part in (0, 1):
            where = [part * 16 * R + at[i]]
            if fmt == "nvfp4":
                where.append(32 * R + part * D + np.arange(D // 16) * 16 + i)
            if fmt in ("fp8", "nvfp4"):
                where.append(np.array([shape[3] - 32 + 16 * part + i]))
            own[slot // page, :, slot % page // 16, np.concatenate(where)] = True
    return own


@pytest.mark.parametrize("fmt", ["bf16", "fp16", "fp8", "nvfp4"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,H,page", [(1, 1, 16), (23, 3, 48), (700, 8, 64)])
def test_other_slots_keep_their_bytes(fmt, D, T, H, page):
    """A write changes no byte but those of its slots; neighbours in the same record, line and 16-byte piece among them."""
    k, v = tokens(T, H, D, "bf16", 1), tokens(T, H, D, "bf16", 2)
    pages = T // page + 3
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(5))[:T].to(torch.int32)
    own = bytes_of(slots.tolist(), H, fmt, D, page, (pages, H, page // 16, KV.record_bytes(fmt, D)))
    for fill in (0xA5, 0x5A):
        data, c = new_cache(fmt, D, H, pages, page, fill=fill)
        moe.moe_kv_write(k, v, slots.cuda(), c, ws_status())
        assert (data.cpu().numpy()[~own] == fill).all()


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_values_of_32_bits(fmt, D):
    """Genuine fp32 inputs, of many sizes, byte by byte."""
    T, H, page = 40, 2, 32
    g = torch.Generator().manual_seed(11)
    k, v = (torch.randn(T, H, D, generator=g) * torch.exp(8 * torch.randn(T, H, 1, generator=g)) for _ in range(2))
    v *= torch.exp(3 * torch.randn(T, H, D, generator=g))
    data, c = new_cache(fmt, D, H, T // page + 1, page)
    slots = torch.arange(T, dtype=torch.int32)
    moe.moe_kv_write(k.cuda(), v.cuda(), slots.cuda(), c, ws_status())
    check_written(data, slots, k, v, fmt, page)


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("step", [-1, 0, 1])
def test_values_of_32_bits_next_to_ties(fmt, step):
    """Values halfway between two codes (and block maxima halfway between two block scales), and one fp32 step to
    either side, where a quotient that is rounded first could land on the tie."""
    D, e4m3 = 64, KV._E4M3
    ties = (e4m3[1:] + e4m3[:-1]) / 2

    def beside(x):
        x = np.asarray(x, dtype=np.float32)
        return x if step == 0 else np.nextafter(x, np.float32(step * np.inf))
    rows = []
    if fmt == "fp8":
        for at in range(0, len(ties), 32):
            r = np.zeros(D, np.float32)
            t = ties[at:at + 32]
            r[:len(t)] = beside(t)
            r[32:32 + len(t)] = -beside(t)
            r[63] = 448.0 if t.max() < 400 else r[63]
            rows.append(r)
    else:
        mid = (KV._E2M1[1:] + KV._E2M1[:-1]) / 2
        for s in e4m3[1:]:
            r = np.zeros(D, np.float32)
            r[0], r[1:8], r[8:15] = 6 * s, beside(mid * s), -beside(mid * s)   # codes' ties under a scale of s
            r[48] = 2688.0                                                      # row scale 1
            rows.append(r)
        for t in ties[:-1]:
            r = np.zeros(D, np.float32)
            r[0], r[1:8] = beside(6 * t), 6 * t * np.linspace(0.1, 0.9, 7)      # the block scale's ties
            r[48] = 2688.0
            rows.append(r)
    x = torch.from_numpy(np.stack(rows))[:, None]
    T = x.shape[0]
    data, c = new_cache(fmt, D, 1, T // 16 + 1, 16)
    slots = torch.arange(T, dtype=torch.int32)
    moe.moe_kv_write(x.cuda(), -x.cuda(), slots.cuda(), c, ws_status())
    check_written(data, slots, x, -x, fmt, 16)


def test_a_write_past_four_gigabytes_leaves_the_rest():
    D, H, page, pages = 128, 8, 128, 20000
    data, c = new_cache("bf16", D, H, pages, page)
    slots = [0, pages * page - 1, pages * page // 2 + 7, 17]
    k, v = tokens(4, H, D, "bf16", 1), tokens(4, H, D, "bf16", 2)
    moe.moe_kv_write(k, v, torch.tensor(slots, dtype=torch.int32, device="cuda"), c, ws_status())
    written = sorted({s // page for s in slots})
    own = bytes_of([written.index(s // page) * page + s % page for s in slots], H, "bf16", D, page,
                   (len(written),) + tuple(data.shape[1:]))
    assert (data[written].cpu().numpy()[~own] == 0).all()
    check_written(data[written], torch.tensor([written.index(s // page) * page + s % page for s in slots]), k, v, "bf16",
                  page)
    for lo, hi in zip([-1] + written, written + [pages]):
        assert not data[lo + 1:hi].any()
