"""Many tokens: four rows of keys and values a lane in the fused cache write, 16 tokens a CTA in the rotation. Bit for bit
what the same calls give for a few tokens at a time (one row a lane), and against float64."""
import pytest
import torch

import bit_block_scaled_gb300 as moe
from gpu_helpers import built, ws_status
from test_front_sizes import ROTATIONS, WRITES
from test_gpu_rope import cache_of, close, make, positions, reference

pytestmark = pytest.mark.gpu
FEW = 700


@pytest.fixture(scope="module", autouse=True)
def lib():
    return built()


@pytest.mark.parametrize("fmt,dtype", [("fp8", torch.bfloat16), ("nvfp4", torch.bfloat16), ("bf16", torch.float32), ("nvfp4", torch.float16)])
@pytest.mark.parametrize("layout,off", [("half", 0), ("interleaved", 0), ("half", 28), ("interleaved", 28)])
@pytest.mark.parametrize("T,hk,D", WRITES)
def test_write(T, hk, D, layout, off, fmt, dtype):
    hq, page = 2, 48
    r, pos = moe.rope(D - off, layout, 150000.0), positions(T)
    qkv = make(T, hq + 2 * hk, D, dtype, T)
    q, k, v = qkv.split((hq, hk, hk), dim=1)
    pages = T // page + 3
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(T))[:T].to(torch.int32).cuda()
    slots[::97] = -1
    slots[T - 1] = -1
    ws = ws_status()
    data, c = cache_of(fmt, pages, page, hk, D)
    out = torch.full((T, hq, D), 7.0, dtype=dtype, device="cuda")
    moe.moe_rope_kv_write(r, pos, q, out, k, v, slots, c, ws)
    few, cf = cache_of(fmt, pages, page, hk, D)
    want = torch.empty_like(out)
    for t in range(0, T, FEW):
        s = slice(t, min(t + FEW, T))
        moe.moe_rope_kv_write(r, pos[s], q[s], want[s], k[s], v[s], slots[s], cf, ws)
    assert torch.equal(data, few) and torch.equal(out, want)
    # and the two calls apart
    kr = torch.empty(T, hk, D, device="cuda")
    moe.moe_rope(r, pos, k.float(), kr)
    plain, cp = cache_of(fmt, pages, page, hk, D)
    moe.moe_kv_write(kr, v.float(), slots, cp, ws)
    assert torch.equal(data, plain)
    # and no query
    again, ca = cache_of(fmt, pages, page, hk, D)
    moe.moe_rope_kv_write(r, pos, None, None, k, v, slots, ca, ws)
    assert torch.equal(again, data) and moe.moe_read_status(ws) == 0


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,hq,hk,D,rot", ROTATIONS)
@pytest.mark.parametrize("pad", [0, 3])
def test_rope(T, hq, hk, D, rot, pad, layout):
    r, pos = moe.rope(rot, layout), positions(T)
    q, k = make(T, hq, D, torch.bfloat16), make(T, hk, D, torch.bfloat16, 1)
    qo = torch.zeros(T, hq, D + pad, dtype=torch.bfloat16, device="cuda")[..., :D]  # pad 3: off the 16-byte grid
    ko = torch.zeros(T, hk, D + pad, dtype=torch.bfloat16, device="cuda")[..., :D]
    moe.moe_rope(r, pos, q, qo, k, ko)
    close(qo, q, reference(q, pos, r, layout), torch.bfloat16, rot)
    close(ko, k, reference(k, pos, r, layout), torch.bfloat16, rot)
    few = torch.zeros_like(q)
    for t in range(0, T, FEW):
        s = slice(t, min(t + FEW, T))
        moe.moe_rope(r, pos[s], q[s], few[s])
    assert torch.equal(qo, few)
