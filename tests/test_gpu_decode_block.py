"""examples/decode_block.py: every stage of a block's step against its oracle on that stage's own inputs, and the
captured step against the eager one."""
import os
import sys

import numpy as np
import pytest
import torch

import bit_block_scaled_gb300 as moe
from gpu_helpers import OL, assert_close, built, get_config, to_numpy
from oracle import group_routing as GR
from oracle import kvcache as KV
from oracle import seam as S

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    return built()


def f64(t):
    return t.double().cpu().numpy()


def block_of(fmt, seed=0):
    from decode_block import DecodeBlock
    b = DecodeBlock(get_config("c0"), fmt=fmt, seed=seed)
    b.h.copy_(torch.randn(b.B, b.cfg.H, generator=torch.Generator().manual_seed(seed + 9)))
    return b


@pytest.mark.parametrize("fmt", ["nvfp4", "fp8", "bf16"])
def test_stages(fmt):
    b = block_of(fmt)
    half = 2.0 ** -8  # of a bf16 result
    for step in range(19):  # past a page of 16
        h0 = f64(b.h)
        b.step()
        assert moe.moe_read_status(b.ws) == 0
        if step not in (0, 15, 18):
            continue
        w = [f64(x) for x in b.norm_w]
        ref = S.norm(h0, "rms", w[0])[0]
        assert np.all(np.abs(f64(b.x) - ref) <= half * np.abs(ref) + 1e-5)
        keys, vals = KV.values(b.data.cpu().numpy(), fmt, b.head_dim)
        out, _, mag, _, _ = KV.attend(f64(b.qkv)[:, :b.q_heads], keys, vals, b.table.cpu().numpy(), b.lens.cpu().numpy(),
                                      b.head_dim ** -0.5, 0, f64(b.sinks))
        # an output's rounding and those of the probabilities, and 2^-10 of the sum for the scores' own
        assert np.all(np.abs(f64(b.q_out) - out) <= half * np.abs(out) + (half + 2.0 ** -10) * mag)
        ids, tw = GR.route_grouped(f64(b.logits), f64(b.sel_bias), b.cfg.k, "sigmoid", 4, 2, "top2")
        assert np.array_equal(b.ids.cpu().numpy(), ids)
        np.testing.assert_allclose(b.tw.cpu().numpy(), tw, rtol=3e-6)
        n = to_numpy({"x": b.mlp_in, "w13": b.w13, "w2": b.w2})
        exp = OL.moe_forward(n["x"], None, n["w13"], n["w2"], b.cfg.k, topk_ids=ids, topk_weights=tw.astype(np.float32))
        assert_close(b.mlp_out.float().cpu().numpy(), exp["out"], "experts")
        o = f64(b.q_out.view(b.B, -1) @ b.w_o.t())
        h1, x1 = S.residual_norm(o, h0, None, None, 1.0, dict(kind="rms", weight=w[1]))
        assert np.all(np.abs(f64(b.mlp_in) - x1) <= half * np.abs(x1) + 1e-5)
        h2, _ = S.residual_norm(f64(b.mlp_out), h1, None, dict(kind="rms", weight=w[2]), 1.0, None)
        assert np.all(np.abs(f64(b.h) - h2) <= 1e-5 * (1 + np.abs(h2)))


def test_captured_step_repeats_the_eager_one():
    a, b = block_of("nvfp4", 3), block_of("nvfp4", 3)
    for _ in range(5):
        a.step()
    b.step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        b.step()
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.lens, b.lens) and torch.equal(a.data, b.data)
    assert torch.equal(a.h, b.h)
