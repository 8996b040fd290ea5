"""Host-side argument checks of the calls around the layer: each call is rejected, or has nothing to do, before
its first CUDA call, so the tests run on the CPU with host buffers standing in for device pointers."""
import pytest
import torch

import bit_block_scaled_gb300 as moe
from bit_block_scaled_gb300 import build as B
from oracle import kvcache as KV

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 6
bf16 = torch.bfloat16


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


def _route(T=4, E=16, k=2, logits=None, bias=None, ids=None, w=None, ws=None, **r):
    logits = torch.zeros(T, E) if logits is None else logits
    moe.moe_route_grouped(logits, bias, k, moe.router(**r), torch.zeros(T, max(k, 1), dtype=torch.int32) if ids is None
                          else ids, torch.zeros(T, max(k, 1)) if w is None else w, _ws() if ws is None else ws, 0)


@pytest.mark.parametrize("kw", [
    dict(k=0, ids=torch.zeros(0, dtype=torch.int32), w=torch.zeros(0)), dict(k=9), dict(E=300, k=2), dict(E=4, k=5),
    dict(score=2), dict(group_score=5), dict(n_group=3), dict(n_group=0), dict(n_group=4, topk_group=0),
    dict(n_group=4, topk_group=5), dict(n_group=8, topk_group=1, k=3),              # k past the kept groups' experts
    dict(n_group=16, topk_group=4, group_score="top2"),                             # groups of one expert
    dict(E=64, n_group=64, topk_group=64), dict(scale=float("nan")),
    dict(logits=torch.zeros(4, 16, dtype=torch.float64)), dict(bias=torch.zeros(15)),
    dict(bias=torch.zeros(16, dtype=bf16)), dict(ids=torch.zeros(4, 2, dtype=torch.int64)), dict(w=torch.zeros(4, 1)),
    dict(logits=torch.zeros(16, 4).t()), dict(logits=torch.zeros(4, 20)[:, 1:17]),   # columns apart, misaligned
    dict(logits=torch.zeros(4, 1).expand(4, 16)), dict(ws=_ws()[1:]),
])
def test_route_rejections(kw):
    assert _code(lambda: _route(**kw)) == INVALID


def test_nothing_to_do():
    _route(T=0)
    x = torch.zeros(0, 64, dtype=bf16)
    moe.moe_residual_norm(x, x, None, None, 1.0, x.clone(), None, None, 0)
    data = torch.zeros(2, 1, 1, KV.record_bytes("fp8", 64), dtype=torch.uint8)
    c = moe.kv_cache(data, "fp8", 64)
    kv = torch.zeros(0, 1, 64)
    none = torch.zeros(0, dtype=torch.int32)
    moe.moe_kv_write(kv, kv, none, c, _ws(), 0)
    moe.moe_kv_read(c, none, kv, kv.clone(), _ws(), 0)
    q = torch.zeros(0, 4, 64, dtype=bf16)
    moe.moe_attn_decode(q, c, torch.zeros(0, 2, dtype=torch.int32), none, q.clone(),
                        _ws(moe.moe_attn_workspace_size(4, 1, 64)), stream=0)
    assert moe.moe_last_launch_count() == 0


def _norm(T=4, H=64, act=bf16, res=None, z="z", r="r", gate=None, post=None, pre=None, h="h", y=None):
    res = act if res is None else res
    mk = lambda v, d: torch.zeros(T, H, dtype=d) if isinstance(v, str) else v  # noqa: E731
    moe.moe_residual_norm(mk(z, act), mk(r, res), gate, post, 1.0, mk(h, res), pre, mk(y, act), 0)


@pytest.mark.parametrize("kw", [
    dict(H=16392), dict(act=bf16, res=torch.float16), dict(act=torch.float32, res=bf16), dict(act=torch.float64),
    dict(y="y"), dict(pre=moe.norm("rms")), dict(h=None), dict(z=None, post=moe.norm("rms")),
    dict(z=None, r=None), dict(post=moe.norm(7)), dict(post=moe.norm("rms", eps=-1.0)),
    dict(post=moe.norm("rms", torch.ones(63))), dict(gate=torch.zeros(4, 64)), dict(gate=torch.zeros(3, 64, dtype=bf16)),
    dict(gate=torch.zeros(4, 128, dtype=bf16)[:, ::2]), dict(z=torch.zeros(4, 72, dtype=bf16)[:, 1:65]),
    dict(h=torch.zeros(1, 64, dtype=bf16).expand(4, 64)), dict(z=torch.zeros(4, 60, dtype=bf16)),
])
def test_norm_rejections(kw):
    assert _code(lambda: _norm(**kw)) == INVALID


def test_norm_parameters_of_two_types():
    assert _code(lambda: moe.norm("layer", torch.ones(8), torch.ones(8, dtype=bf16))) == INVALID


@pytest.mark.parametrize("fmt", ["bf16", "fp16", "fp8", "nvfp4"])
def test_record_bytes(fmt):
    for D in (64, 128, 256):
        assert moe.moe_kv_record_bytes(fmt, D) == KV.record_bytes(fmt, D)
    assert moe.moe_kv_record_bytes(fmt, 96) == 0 and moe.moe_kv_record_bytes(9, 64) == 0


def _cache(fmt="fp8", D=64, H=2, pages=2, per=1):
    return torch.zeros(pages, H, per, KV.record_bytes(fmt, D), dtype=torch.uint8)


def _write(data=None, fmt="fp8", D=64, T=3, k=None, slots=None, edit=None, ws=None, read=False):
    data = _cache(fmt, D) if data is None else data
    c = moe.kv_cache(data, fmt, D)
    if edit:
        edit(c)
    k = torch.zeros(T, 2, D, dtype=bf16) if k is None else k
    slots = torch.zeros(T, dtype=torch.int32) if slots is None else slots
    if read:
        moe.moe_kv_read(c, slots, k, k.clone(), _ws() if ws is None else ws, 0)
    else:
        moe.moe_kv_write(k, k, slots, c, _ws() if ws is None else ws, 0)


@pytest.mark.parametrize("read", [False, True])
@pytest.mark.parametrize("kw", [
    dict(k=torch.zeros(3, 2, 63, dtype=bf16)), dict(k=torch.zeros(3, 2, 64, dtype=torch.float64)),
    dict(k=torch.zeros(3, 2, 128, dtype=bf16)[:, :, ::2]), dict(k=torch.zeros(3, 2, 68, dtype=bf16)[:, :, :64]),
    dict(slots=torch.zeros(3, dtype=torch.int64)), dict(ws=_ws()[8:]),
    dict(edit=lambda c: setattr(c, "page_size", 24)), dict(edit=lambda c: setattr(c, "page_size", 8192)),
    dict(edit=lambda c: setattr(c, "num_pages", 1 << 28)), dict(edit=lambda c: setattr(c, "num_pages", 0)),
    dict(edit=lambda c: setattr(c, "data", 0)), dict(edit=lambda c: setattr(c, "fmt", 4)),
])
def test_cache_rejections(read, kw):
    assert _code(lambda: _write(read=read, **kw)) == INVALID


def test_overlapping_outputs_are_refused():
    assert _code(lambda: _write(k=torch.zeros(1, 2, 64, dtype=bf16).expand(3, 2, 64), read=True)) == INVALID


def test_cache_views():
    assert _code(lambda: moe.kv_cache(_cache().float(), "fp8", 64)) == INVALID
    assert _code(lambda: moe.kv_cache(_cache()[:, :, :, :-1], "fp8", 64)) == INVALID
    assert _code(lambda: moe.kv_cache(_cache(), "nvfp4", 64)) == INVALID
    c = moe.kv_cache(torch.zeros(1, 1, 1, 5, dtype=torch.uint8), "fp8", 96)
    q = torch.zeros(1, 1, 96, dtype=bf16)
    assert _code(lambda: moe.moe_kv_write(q, q, torch.zeros(1, dtype=torch.int32), c, _ws(), 0)) == UNSUPPORTED


def _attn(fmt="fp8", D=64, B=2, heads=4, q=None, out=None, table=None, lens=None, ws=None, edit=None, **kw):
    c = moe.kv_cache(_cache(fmt, D), fmt, D)
    if edit:
        edit(c)
    q = torch.zeros(B, heads, D, dtype=bf16) if q is None else q
    moe.moe_attn_decode(q, c, torch.zeros(B, 2, dtype=torch.int32) if table is None else table,
                        torch.zeros(B, dtype=torch.int32) if lens is None else lens,
                        torch.zeros_like(q) if out is None else out,
                        _ws(moe.moe_attn_workspace_size(4, 2, 64) * 4) if ws is None else ws, stream=0, **kw)


@pytest.mark.parametrize("kw,code", [
    (dict(heads=3), INVALID), (dict(heads=512), INVALID), (dict(window=-1), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(ws=_ws()), WORKSPACE), (dict(fmt="bf16", q=torch.zeros(2, 4, 64, dtype=torch.float16)), UNSUPPORTED),
    (dict(fmt="fp16"), UNSUPPORTED), (dict(q=torch.zeros(2, 4, 64)), INVALID),
    (dict(q=torch.zeros(2, 4, 68, dtype=bf16)[:, :, :64]), INVALID), (dict(lens=torch.zeros(2, dtype=torch.int64)), INVALID),
    (dict(lens=torch.zeros(3, dtype=torch.int32)), INVALID), (dict(sinks=torch.zeros(3)), INVALID),
    (dict(lse=torch.zeros(2, 4, dtype=bf16)), INVALID), (dict(table=torch.zeros(2, 2, dtype=torch.int64)), INVALID),
    (dict(table=torch.zeros(2, 2, dtype=torch.int32).t()), INVALID), (dict(B=5000), UNSUPPORTED),
    (dict(out=torch.zeros(1, 4, 64, dtype=bf16).expand(2, 4, 64)), INVALID),
    (dict(out=torch.zeros(2, 1, 64, dtype=bf16).expand(2, 4, 64)), INVALID),
    (dict(out=torch.zeros(2, 4, 64)), INVALID), (dict(edit=lambda c: setattr(c, "page_size", 20)), INVALID),
])
def test_attention_rejections(kw, code):
    assert _code(lambda: _attn(**kw)) == code


def test_attention_workspace():
    assert moe.moe_attn_workspace_size(64, 8, 128) > 0
    assert _code(lambda: moe.moe_attn_workspace_size(7, 2, 128)) == INVALID
    assert _code(lambda: moe.moe_attn_workspace_size(8, 2, 80)) == UNSUPPORTED


def test_host_tensors_need_a_stream_that_says_so():
    """Without a stream the tensors' device gives it: host tensors are refused there, not launched on."""
    x = torch.zeros(4, 64, dtype=bf16)
    assert _code(lambda: moe.moe_residual_norm(x, x, None, None, 1.0, x, None, None)) == INVALID
    assert _code(lambda: moe.moe_route_grouped(torch.zeros(2, 8), None, 2, moe.router(),
                                               torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2), _ws())) == INVALID


def test_arguments_of_another_kind():
    assert _code(lambda: moe.moe_residual_norm([1], None, None, None, 1.0, None, None, None, 0)) == INVALID
    assert _code(lambda: _norm(z=torch.zeros(4, 64, dtype=bf16), post="rms")) == INVALID
    assert _code(lambda: _route(ws=_ws(16))) == INVALID
    x = torch.zeros(2, 64, dtype=bf16)
    assert _code(lambda: moe.moe_residual_norm(x, x, None, None, "one", x, None, None, 0)) == INVALID
    assert _code(lambda: moe.moe_residual_norm(x, x, None, None, 1.0, x, None, None, "stream")) == INVALID


def _strided(shape, strides, dtype=bf16):
    return torch.zeros(4096, dtype=dtype).as_strided(shape, strides)


@pytest.mark.parametrize("strides", [(64, 64), (64, 128), (128, 64 + 8), (8, 1024), (256, 0), (0, 64), (160, 128),
                                     (128, 160)])
def test_outputs_whose_rows_meet_are_refused(strides):
    """Rows (token, head) of three tokens and three heads that share elements would be written by two lanes."""
    x = _strided((3, 3, 64), strides + (1,))
    c = moe.kv_cache(torch.zeros(1, 3, 1, KV.record_bytes("fp8", 64), dtype=torch.uint8), "fp8", 64)
    slots = torch.zeros(3, dtype=torch.int32)
    for k, v in ((x, None), (None, x)):
        assert _code(lambda: moe.moe_kv_read(c, slots, k, v, _ws(), 0)) == INVALID
    q = torch.zeros(3, 3, 64, dtype=bf16)
    assert _code(lambda: moe.moe_attn_decode(q, c, torch.zeros(3, 2, dtype=torch.int32), slots, x,
                                             _ws(moe.moe_attn_workspace_size(3, 3, 64)), stream=0)) == INVALID
