"""Host-side argument checks of the batch plan, of rotary positions and of 4-bit operands: each call is rejected, or has
nothing to do, before its first CUDA call, so the tests run on the CPU with host buffers standing in for device pointers."""
import pytest
import torch

import bit_block_scaled_gb300 as moe
from bit_block_scaled_gb300 import build as B
from oracle import kvcache as KV

INVALID, UNSUPPORTED = 1, 2
bf16, i32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return moe.load()


def _code(fn):
    with pytest.raises(moe.MoeError) as e:
        fn()
    return e.value.code


def _ws(n=256):
    return torch.zeros(n, dtype=torch.uint8)


def ints(*shape):
    return torch.zeros(shape, dtype=i32)


# ------------------------------------------------------------------------------------------------- plan
def _plan(B=4, T=8, pages=10, cols=3, page=16, **kw):
    a = dict(new=ints(B), lens=ints(B), table=ints(B, cols), free=ints(pages), count=ints(1), slots=ints(T), out=ints(B),
             left=ints(1), ws=_ws(), positions=ints(T), seqs=ints(T), offsets=ints(B + 1))
    a.update(kw)
    moe.moe_batch_plan(a["new"], a["lens"], a["table"], a["free"], a["count"], page, a["slots"], a["out"], a["left"], a["ws"],
                       positions=a["positions"], seq_ids=a["seqs"], offsets=a["offsets"], stream=0)


@pytest.mark.parametrize("kw", [
    dict(page=0), dict(page=24), dict(page=8192), dict(pages=0), dict(new=ints(3)), dict(lens=torch.zeros(4, dtype=torch.int64)),
    dict(table=ints(3, 3)), dict(table=ints(4, 3).long()), dict(table=ints(3, 4).t()), dict(table=ints(12)), dict(count=ints(2)),
    dict(left=ints(0)), dict(out=ints(5)), dict(positions=ints(7)), dict(seqs=torch.zeros(8)), dict(offsets=ints(4)),
    dict(slots=torch.zeros(8, dtype=torch.int64)), dict(ws=_ws()[8:]), dict(ws=_ws(16)), dict(ws=None), dict(new=None),
    dict(free=None), dict(table=ints(1, 3).expand(4, 3)), dict(new=[1, 2, 3, 4])])
def test_plan_rejections(kw):
    assert _code(lambda: _plan(**kw)) == INVALID


def test_plan_sizes():
    assert _code(lambda: _plan(B=4097)) == UNSUPPORTED
    assert _code(lambda: _plan(cols=1 << 17, page=4096, B=4096, table=ints(1, 1).expand(4096, 1 << 19))) == INVALID
    lib, P = moe.load(), 1 << 20  # nothing is read
    args = [P, P, 4, 16, 1 << 27, P, 100, 100, P, P, P, P, P, 8, 0, P, P, P, P, None]
    assert lib.moe_batch_plan(*args) == INVALID  # slots past 31 bits
    args[4] = 100
    for at in (0, 1, 5, 8, 9, 10, 11, 15, 18):
        for bad in (None, P + 2):
            a = list(args)
            a[at] = bad
            assert lib.moe_batch_plan(*a) == INVALID, at
    a = list(args)
    a[13] = (1 << 28) + 1
    assert lib.moe_batch_plan(*a) == INVALID
    a = list(args)
    a[6] = 99  # rows of the table that overlap
    assert lib.moe_batch_plan(*a) == INVALID
    a = list(args)
    a[14] = -1
    assert lib.moe_batch_plan(*a) == INVALID


def test_nothing_to_do():
    none = ints(0)
    moe.moe_batch_plan(none, none, ints(0, 4), ints(4), ints(1), 16, none, none, ints(1), _ws(), stream=0)
    x = torch.zeros(0, 2, 64, dtype=bf16)
    r = moe.rope(64, device="cpu")
    moe.moe_rope(r, none, x, x.clone(), stream=0)
    c = moe.kv_cache(torch.zeros(2, 2, 1, KV.record_bytes("fp8", 64), dtype=torch.uint8), "fp8", 64)
    moe.moe_rope_kv_write(r, none, None, None, x, x, none, c, _ws(), 0)
    f = _fp4(0, 64)
    moe.moe_fp4_quantize(torch.zeros(0, 64), f, 0)
    moe.moe_fp4_dequantize(f, torch.zeros(0, 64), 0)
    moe.moe_fp4_linear(f, _fp4(8, 64), None, torch.zeros(0, 8), _ws(), 0)
    moe.moe_fp4_pack_scales(torch.zeros(0, 4, dtype=torch.uint8), "nvfp4", 64, torch.zeros(0, dtype=torch.uint8), 0)
    assert moe.moe_last_launch_count() == 0


# ------------------------------------------------------------------------------------------------- rope
def _rope(T=4, D=64, rot=64, q=None, qo=None, k=None, ko=None, pos=None, edit=None, stream=0):
    r = moe.rope(rot, device="cpu")
    if edit:
        edit(r)
    q = torch.zeros(T, 3, D, dtype=bf16) if q is None else q
    moe.moe_rope(r, ints(T) if pos is None else pos, q, torch.zeros_like(q) if qo is None else qo, k, ko, stream)


x4 = torch.zeros(4, 3, 64, dtype=bf16)


@pytest.mark.parametrize("kw", [
    dict(D=512, rot=64), dict(rot=66), dict(edit=lambda r: setattr(r, "rot_dim", 3)), dict(edit=lambda r: setattr(r, "rot_dim", 0)),
    dict(edit=lambda r: setattr(r, "layout", 2)), dict(edit=lambda r: setattr(r, "turns", 0)),
    dict(edit=lambda r: setattr(r, "turns", r.turns + 4)), dict(edit=lambda r: setattr(r, "amplitude", float("nan"))),
    dict(edit=lambda r: setattr(r, "amplitude", 1e300)),
    dict(edit=lambda r: setattr(r, "place", 1)), dict(pos=ints(3)), dict(pos=torch.zeros(4, dtype=torch.int64)),
    dict(q=torch.zeros(4, 3, 64, dtype=torch.float64)), dict(q=x4, qo=torch.zeros(4, 3, 64)), dict(q=x4, qo=x4[:, :2]),
    dict(k=x4), dict(ko=x4), dict(k=x4, ko=torch.zeros(4, 2, 64, dtype=bf16)), dict(k=torch.zeros(4, 2, 64), ko=torch.zeros(4, 2, 64)),
    dict(q=torch.zeros(4, 3, 128, dtype=bf16)[..., ::2]), dict(q=torch.zeros(4, 192, dtype=bf16)),
    dict(q=x4, qo=torch.zeros(1, 3, 64, dtype=bf16).expand(4, 3, 64)), dict(q=x4, qo=torch.zeros(4, 1, 64, dtype=bf16).expand(4, 3, 64)),
    dict(q=x4, qo=x4.reshape(-1)[:768].as_strided((4, 3, 64), (64, 256, 1))),  # its own memory in another order
    dict(stream=None), dict(stream="s")])
def test_rope_rejections(kw):
    assert _code(lambda: _rope(**kw)) == INVALID


def _write(T=3, D=64, q=None, qo=None, k=None, v=None, slots=None, pos=None, fmt="fp8", edit=None, ws=None, rot=64):
    c = moe.kv_cache(torch.zeros(2, 2, 1, KV.record_bytes(fmt, D), dtype=torch.uint8), fmt, D)
    r = moe.rope(rot, device="cpu")
    if edit:
        edit(c)
    k = torch.zeros(T, 2, D, dtype=bf16) if k is None else k
    moe.moe_rope_kv_write(r, ints(T) if pos is None else pos, q, qo, k, k if v is None else v, ints(T) if slots is None else slots,
                          c, _ws() if ws is None else ws, 0)


x3 = torch.zeros(3, 4, 64, dtype=bf16)


@pytest.mark.parametrize("kw", [
    dict(k=torch.zeros(3, 2, 63, dtype=bf16)), dict(k=torch.zeros(3, 2, 64, dtype=torch.float64)), dict(v=torch.zeros(3, 2, 64)),
    dict(k=torch.zeros(3, 2, 68, dtype=bf16)[..., :64]), dict(k=torch.zeros(4, 2, 64, dtype=bf16)), dict(pos=ints(2)),
    dict(slots=torch.zeros(3, dtype=torch.int64)), dict(ws=_ws()[8:]), dict(rot=128), dict(q=x3), dict(qo=x3),
    dict(q=x3, qo=torch.zeros(3, 4, 64)), dict(q=torch.zeros(3, 4, 64), qo=torch.zeros(3, 4, 64)),
    dict(q=torch.zeros(3, 4, 68, dtype=bf16)[..., :64], qo=x3), dict(q=x3, qo=torch.zeros(1, 4, 64, dtype=bf16).expand(3, 4, 64)),
    dict(edit=lambda c: setattr(c, "page_size", 24)), dict(edit=lambda c: setattr(c, "data", 0)),
    dict(edit=lambda c: setattr(c, "fmt", 9))])
def test_rope_write_rejections(kw):
    assert _code(lambda: _write(**kw)) == INVALID


# ------------------------------------------------------------------------------------------------- 4 bits
def _fp4(rows=4, K=64, fmt="nvfp4", row_scale="r"):
    r = torch.zeros(rows) if isinstance(row_scale, str) and fmt == "nvfp4" else None if isinstance(row_scale, str) else row_scale
    return moe.fp4(torch.zeros(rows, K // 2, dtype=torch.uint8), torch.zeros(moe.moe_fp4_scale_bytes(fmt, rows, K), dtype=torch.uint8),
                   fmt, r)


def test_scale_bytes():
    assert moe.moe_fp4_scale_bytes("nvfp4", 1, 32) == 512 and moe.moe_fp4_scale_bytes("mxfp4", 129, 160) == 2 * 2 * 512
    assert moe.moe_fp4_scale_bytes("nvfp4", 128, 2880) == 45 * 512 and moe.moe_fp4_scale_bytes("nvfp4", 0, 64) == 0
    for bad in (("int4", 4, 64), ("nvfp4", 4, 48), ("nvfp4", 4, 0), ("nvfp4", -1, 64), ("mxfp4", 1 << 24, 64), ("mxfp4", 4, (1 << 20) + 32)):
        assert moe.moe_fp4_scale_bytes(*bad) == 0


u8 = torch.uint8


@pytest.mark.parametrize("fn", [
    lambda: moe.fp4(torch.zeros(4, 32), torch.zeros(512, dtype=u8), "nvfp4"),
    lambda: moe.fp4(torch.zeros(4, 64, dtype=u8)[:, :32], torch.zeros(512, dtype=u8), "nvfp4"),
    lambda: moe.fp4(torch.zeros(4, 32, dtype=u8), torch.zeros(511, dtype=u8), "nvfp4"),
    lambda: moe.fp4(torch.zeros(4, 32, dtype=u8), torch.zeros(512), "nvfp4"),
    lambda: moe.fp4(torch.zeros(4, 24, dtype=u8), torch.zeros(0, dtype=u8), "nvfp4"),
    lambda: moe.fp4(torch.zeros(4, 32, dtype=u8), torch.zeros(512, dtype=u8), "nvfp4", torch.zeros(3)),
    lambda: moe.fp4(torch.zeros(4, 32, dtype=u8), torch.zeros(512, dtype=u8), "nvfp4", torch.zeros(4, dtype=bf16)),
    lambda: moe.fp4(torch.zeros(128, dtype=u8), torch.zeros(512, dtype=u8), "nvfp4")])
def test_matrices(fn):
    assert _code(fn) == INVALID


def edited(f, **kw):
    for k, v in kw.items():
        setattr(f, k, v)
    return f


@pytest.mark.parametrize("fn", [
    lambda: moe.moe_fp4_quantize(torch.zeros(3, 64), _fp4(), 0), lambda: moe.moe_fp4_quantize(torch.zeros(4, 32), _fp4(), 0),
    lambda: moe.moe_fp4_quantize(torch.zeros(4, 64, dtype=torch.float64), _fp4(), 0),
    lambda: moe.moe_fp4_quantize(torch.zeros(4, 68)[:, :64], _fp4(), 0), lambda: moe.moe_fp4_quantize(torch.zeros(64, 4).t(), _fp4(), 0),
    lambda: moe.moe_fp4_quantize(torch.zeros(4, 64), _fp4(row_scale=None), 0),
    lambda: moe.moe_fp4_quantize(torch.zeros(4, 64), _fp4(row_scale=torch.zeros(1)), 0),
    lambda: moe.moe_fp4_quantize(torch.zeros(4, 64), _fp4(), None), lambda: moe.moe_fp4_quantize(None, _fp4(), 0),
    lambda: moe.moe_fp4_quantize(torch.zeros(4, 64), None, 0), lambda: moe.moe_fp4_quantize(torch.zeros(4, 64), edited(_fp4(), q=0), 0),
    lambda: moe.moe_fp4_quantize(torch.zeros(4, 64), edited(_fp4(), fmt=2), 0),
    lambda: moe.moe_fp4_quantize(torch.zeros(4, 64), edited(_fp4(), place=1), 0),
    lambda: moe.moe_fp4_dequantize(_fp4(), torch.zeros(4, 32), 0), lambda: moe.moe_fp4_dequantize(_fp4(), torch.zeros(1, 64).expand(4, 64), 0),
    lambda: moe.moe_fp4_dequantize(_fp4(), torch.zeros(4, 68)[:, :64], 0),
    lambda: moe.moe_fp4_dequantize(edited(_fp4("nvfp4" and 4), row_scale_stride=2), torch.zeros(4, 64), 0),
    lambda: moe.moe_fp4_pack_scales(torch.zeros(4, 3, dtype=u8), "nvfp4", 64, torch.zeros(512, dtype=u8), 0),
    lambda: moe.moe_fp4_pack_scales(torch.zeros(4, 4, dtype=u8), "nvfp4", 64, torch.zeros(500, dtype=u8), 0),
    lambda: moe.moe_fp4_pack_scales(torch.zeros(4, 4), "nvfp4", 64, torch.zeros(512, dtype=u8), 0),
    lambda: moe.moe_fp4_linear(_fp4(), _fp4(8), None, torch.zeros(4, 7), _ws(), 0),
    lambda: moe.moe_fp4_linear(_fp4(), _fp4(8, 96), None, torch.zeros(4, 8), _ws(), 0),
    lambda: moe.moe_fp4_linear(_fp4(), _fp4(8, fmt="mxfp4"), None, torch.zeros(4, 8), _ws(), 0),
    lambda: moe.moe_fp4_linear(_fp4(), _fp4(8), torch.zeros(7), torch.zeros(4, 8), _ws(), 0),
    lambda: moe.moe_fp4_linear(_fp4(), _fp4(8), torch.zeros(8, dtype=bf16), torch.zeros(4, 8), _ws(), 0),
    lambda: moe.moe_fp4_linear(_fp4(), _fp4(8), None, torch.zeros(4, 8, dtype=torch.float64), _ws(), 0),
    lambda: moe.moe_fp4_linear(_fp4(), _fp4(8), None, torch.zeros(1, 8).expand(4, 8), _ws(), 0),
    lambda: moe.moe_fp4_linear(_fp4(), _fp4(8), None, torch.zeros(8, 4).t(), _ws(), 0),
    lambda: moe.moe_fp4_linear(_fp4(), _fp4(8), None, torch.zeros(4, 8), _ws()[8:], 0),
    lambda: moe.moe_fp4_linear(_fp4(), edited(_fp4(8, fmt="mxfp4"), fmt=0, row_scale=3), None, torch.zeros(4, 8), _ws(), 0)])
def test_four_bit_rejections(fn):
    assert _code(fn) == INVALID


def test_rows_too_wide_to_quantise():
    f = _fp4(1, 32800)
    assert _code(lambda: moe.moe_fp4_quantize(torch.zeros(1, 32800), f, 0)) == UNSUPPORTED


def test_structs_keep_their_tensors():
    f = _fp4()
    assert f.tensors[0].data_ptr() == f.q and f.tensors[1].data_ptr() == f.scales
    r = moe.rope(32, device="cpu")
    assert r.table.data_ptr() == r.turns and r.rot_dim == 32
