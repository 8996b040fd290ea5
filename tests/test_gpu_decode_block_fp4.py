"""examples/decode_block.py with 4-bit projections, rotary positions and planned pages: each call's outputs from its own
inputs against its oracle, and the captured step against the eager one."""
import os
import sys

import numpy as np
import pytest
import torch

import bit_block_scaled_gb300 as moe
from gpu_helpers import built, get_config
from oracle import fp4 as F
from oracle import kvcache as KV
from oracle import plan as P
from oracle import rope as R

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8  # of a bf16 result


@pytest.fixture(scope="module", autouse=True)
def lib():
    return built()


def f64(t):
    return t.double().cpu().numpy()


def block_of(fmt, proj, layout, seed=0):
    from decode_block import DecodeBlock
    b = DecodeBlock(get_config("c0"), fmt=fmt, seed=seed, proj=proj,
                    rope=dict(rot_dim=64, layout=layout, scaling="yarn", base=150000.0, factor=32.0))
    b.h.copy_(torch.randn(b.B, b.cfg.H, generator=torch.Generator().manual_seed(seed + 9)))
    return b


def values_of(f, fmt):
    q, s, r = f.tensors
    return F.values(q.cpu().numpy(), F.untile(s.cpu().numpy(), q.shape[0], q.shape[1] * 2 // F.BLOCK[fmt]),
                    None if r is None else f64(r), fmt)


def close(got, ref, mag, K):
    assert np.all(np.abs(got - ref) <= HALF * np.abs(ref) + (K / 64 + 4) * 2.0 ** -22 * (mag + np.abs(ref)))


@pytest.mark.parametrize("fmt,proj,layout", [("nvfp4", "nvfp4", "half"), ("bf16", "mxfp4", "interleaved"), ("fp8", "nvfp4", "half")])
def test_stages(fmt, proj, layout):
    b = block_of(fmt, proj, layout)
    turns = b.rope.table.cpu().numpy().view(np.uint64)
    for step in range(19):  # past a page of 16
        before = [t.cpu().numpy() for t in (b.new_lens, b.lens, b.table, b.free, b.free_count)]
        b.step()
        assert moe.moe_read_status(b.ws) == 0
        plan = P.batch_plan(*before[:4], int(before[4][0]), b.page, b.B, 1)
        for got, name in ((b.slots, "slots"), (b.positions, "positions"), (b.lens, "lens"), (b.table, "table")):
            np.testing.assert_array_equal(got.cpu().numpy(), plan[name])
        if step not in (0, 15, 18):
            continue
        q, s, r = F.quantise_rows(f64(b.x), proj)
        x = F.values(q, s, r, proj)
        np.testing.assert_array_equal(values_of(b.qkv_x, proj), x)
        qkv, mag = F.linear(x, values_of(b.qkv_w, proj))
        qkv, mag = qkv.reshape(b.B, -1, b.head_dim), mag.reshape(b.B, -1, b.head_dim)
        n = b.q_heads
        # keys and values come out of the product and are rotated no further in b.qkv; queries are, in place
        close(f64(b.qkv)[:, n:], qkv[:, n:], mag[:, n:], b.cfg.H)
        a = R.angles(b.positions.cpu().numpy(), turns)
        amp = b.rope.amplitude
        rq = R.rotate(qkv[:, :n], a, layout, amp)
        slack = amp * (HALF * np.abs(qkv[:, :n]).max(axis=2, keepdims=True) * 2 + 1e-5 * mag[:, :n].max(axis=2, keepdims=True))
        assert np.all(np.abs(f64(b.qkv)[:, :n] - rq) <= HALF * np.abs(rq) + slack)
        # the newest keys in the cache are those of b.qkv, rotated
        keys, vals = KV.values(b.data.cpu().numpy(), fmt, b.head_dim)
        rk = R.rotate(f64(b.qkv)[:, n:n + b.kv_heads], a, layout, amp)
        rel = {"bf16": 2.0 ** -8, "fp8": 2.0 ** -4, "nvfp4": 0.25}[fmt]  # of a row's largest value
        slots = b.slots.cpu().numpy()
        held = keys[slots // b.page, :, slots % b.page]
        assert np.all(np.abs(held - rk) <= rel * np.abs(rk).max(axis=2, keepdims=True) + 1e-6)
        out, _, m, _, _ = KV.attend(f64(b.qkv)[:, :n], keys, vals, b.table.cpu().numpy(), b.lens.cpu().numpy(),
                                    b.head_dim ** -0.5, 0, f64(b.sinks))
        assert np.all(np.abs(f64(b.q_out) - out) <= HALF * np.abs(out) + (HALF + 2.0 ** -10) * m)
        q, s, r = F.quantise_rows(f64(b.q_out).reshape(b.B, -1), proj)
        o, mag = F.linear(F.values(q, s, r, proj), values_of(b.o_w, proj))
        close(f64(b.o), o, mag, n * b.head_dim)


@pytest.mark.parametrize("proj", ["nvfp4", "mxfp4"])
def test_captured_step_repeats_the_eager_one(proj):
    a, b = block_of("nvfp4", proj, "half", 3), block_of("nvfp4", proj, "half", 3)
    for _ in range(20):
        a.step()
    b.step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        b.step()
    for _ in range(19):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.lens, b.lens) and torch.equal(a.data, b.data) and torch.equal(a.table, b.table)
    assert torch.equal(a.h, b.h) and moe.moe_read_status(b.ws) == 0


def test_sequences_that_end_give_their_pages_back():
    b = block_of("fp8", "nvfp4", "half", 5)
    for _ in range(17):
        b.step()
    free = int(b.free_count)
    b.new_lens[3] = -1
    b.step()
    assert int(b.lens[3]) == 0 and int(b.free_count) == free + 2 and int(b.slots[3]) == -1
    b.new_lens[3] = 1
    b.step()
    assert int(b.lens[3]) == 1 and int(b.positions[2]) == 18 and int(b.positions[3]) == 0
    assert torch.isfinite(b.h).all() and moe.moe_read_status(b.ws) == 0
