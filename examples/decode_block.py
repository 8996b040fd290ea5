"""One decoder block of an MoE model, decoding: norm, the plan of the step's pages and slots, attention of the newest
token over a quantised paged cache, norm with the residual, grouped routing, the MoE layer's steps, and the residual
again, all in one CUDA graph a token. The dense projections are products of 4-bit operands or plain matrix products,
queries and keys are rotated by their positions or not.

    python examples/decode_block.py            # a small block, 32 tokens for each of 16 sequences

``DecodeBlock.step`` is the sequence of calls that a serving program makes; ``main`` fills the sequences token
by token and prints the time a step takes.
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import bit_block_scaled_gb300 as moe  # noqa: E402
from synth import get_config, make_layer  # noqa: E402


class DecodeBlock:
    """Weights, cache and buffers of one block for B sequences of up to max_tokens tokens each.

    cfg: a layer of synth.configs with T = B; its experts are taken in n_group groups, topk_group of them a
    token, by sigmoid scores with a balancing bias. proj: the dense projections in "bf16", or their weights and
    inputs in "nvfp4" or "mxfp4". rope: arguments of moe.rope(), None for queries and keys as they are."""

    def __init__(self, cfg, q_heads=8, kv_heads=2, head_dim=64, fmt="nvfp4", page=16, max_tokens=64, n_group=4,
                 topk_group=2, seed=0, proj="bf16", rope=None):
        B, H, dev = cfg.T, cfg.H, "cuda"
        self.cfg, self.B, self.q_heads, self.kv_heads, self.head_dim, self.page = cfg, B, q_heads, kv_heads, head_dim, page
        g = torch.Generator().manual_seed(seed)

        def weight(n, k):
            return (torch.randn(n, k, generator=g) * k ** -0.5).to(torch.bfloat16).to(dev)
        self.w_qkv = weight((q_heads + 2 * kv_heads) * head_dim, H)
        self.w_o = weight(H, q_heads * head_dim)
        self.w_router = weight(cfg.E, H)
        self.sel_bias = (torch.randn(cfg.E, generator=g) * 0.1).to(dev)
        self.sinks = torch.randn(q_heads, generator=g).to(dev)
        layer = make_layer(cfg, seed, device=dev)
        self.w13, self.w2 = layer["w13"], layer["w2"]
        self.q13, self.q2 = moe.qweight(self.w13), moe.qweight(self.w2)
        self.norm_w = [(1 + 0.1 * torch.randn(H, generator=g)).to(torch.bfloat16).to(dev) for _ in range(3)]
        # before attention; after it, before the experts; after the experts
        self.n_attn, self.n_mlp, self.n_post = (moe.norm("rms", w, eps=1e-5) for w in self.norm_w)
        self.router = moe.router("sigmoid", n_group, topk_group, "top2", renormalize=True, scale=1.0)
        self.proj, self.rope = proj, None if rope is None else moe.rope(**rope)
        self.qkv_w = self.qkv_x = self.o_w = self.o_x = None
        if proj != "bf16":
            self.qkv_w, self.o_w = self.quantised(self.w_qkv), self.quantised(self.w_o)
            self.qkv_x, self.o_x = self.operand(B, H), self.operand(B, q_heads * head_dim)
        # cache: its pages are on a stack, from which every step takes what it needs
        per_seq = -(-max_tokens // page)
        self.data = torch.zeros(B * per_seq, kv_heads, page // 16, moe.moe_kv_record_bytes(fmt, head_dim),
                                dtype=torch.uint8, device=dev)
        self.cache = moe.kv_cache(self.data, fmt, head_dim)
        self.free = torch.randperm(B * per_seq, generator=g).to(torch.int32).to(dev)
        self.free_count = torch.full((1,), B * per_seq, dtype=torch.int32, device=dev)
        self.table = torch.full((B, per_seq), -1, dtype=torch.int32, device=dev)
        self.lens = torch.zeros(B, dtype=torch.int32, device=dev)
        self.new_lens = torch.ones(B, dtype=torch.int32, device=dev)  # a token for each sequence a step, -1 ends one
        self.slots, self.positions = (torch.empty(B, dtype=torch.int32, device=dev) for _ in range(2))
        self.max_tokens = max_tokens
        # buffers
        bf, i32 = dict(dtype=torch.bfloat16, device=dev), dict(dtype=torch.int32, device=dev)
        self.h = torch.zeros(B, H, device=dev)  # residual stream, fp32
        self.x, self.mlp_in, self.mlp_out = (torch.empty(B, H, **bf) for _ in range(3))
        self.q_out = torch.empty(B, q_heads, head_dim, **bf)
        self.qkv = torch.empty(B, q_heads + 2 * kv_heads, head_dim, **bf)
        self.o = torch.empty(B, H, **bf)
        T, E, k, P = B, cfg.E, cfg.k, moe.moe_padded_rows(B, cfg.k, cfg.E, 16)
        self.ids, self.tw = torch.empty(T, k, **i32), torch.empty(T, k, device=dev)
        self.sorted, self.offsets = torch.empty(P, **i32), torch.empty(E + 1, **i32)
        self.blocks, self.row_pos = torch.empty(P // 16, **i32), torch.empty(T * k, **i32)
        self.x_perm = torch.empty(P, H, **bf)
        self.act, self.y = torch.empty(P, cfg.I, **bf), torch.empty(P, H, **bf)
        self.ws = torch.zeros(moe.moe_attn_workspace_size(q_heads, kv_heads, head_dim), dtype=torch.uint8, device=dev)

    def operand(self, rows, K):
        """Buffers of a 4-bit matrix."""
        return moe.fp4(torch.empty(rows, K // 2, dtype=torch.uint8, device="cuda"),
                       torch.empty(moe.moe_fp4_scale_bytes(self.proj, rows, K), dtype=torch.uint8, device="cuda"), self.proj,
                       torch.empty(rows, device="cuda") if self.proj == "nvfp4" else None)

    def quantised(self, w):
        f = self.operand(*w.shape)
        moe.moe_fp4_quantize(w, f)
        return f

    def project(self, x, w, x4, w4, out):
        """out = x w^T."""
        if self.proj == "bf16":
            torch.mm(x, w.t(), out=out)
        else:
            moe.moe_fp4_quantize(x, x4)
            moe.moe_fp4_linear(x4, w4, None, out, self.ws)

    def step(self):
        """The block on self.h [B, H] (in place), the sequences one token longer. No host synchronisation."""
        cfg, B, D = self.cfg, self.B, self.head_dim
        T, E, k = B, cfg.E, cfg.k
        # attention
        moe.moe_residual_norm(None, self.h, None, None, 1.0, None, self.n_attn, self.x)
        self.project(self.x, self.w_qkv, self.qkv_x, self.qkv_w, self.qkv.view(B, -1))
        q, kk, v = self.qkv.split((self.q_heads, self.kv_heads, self.kv_heads), dim=1)
        moe.moe_batch_plan(self.new_lens, self.lens, self.table, self.free, self.free_count, self.page, self.slots, self.lens,
                           self.free_count, self.ws, positions=self.positions, rows_each=1)
        if self.rope is None:
            moe.moe_kv_write(kk, v, self.slots, self.cache, self.ws)
        else:
            moe.moe_rope_kv_write(self.rope, self.positions, q, q, kk, v, self.slots, self.cache, self.ws)
        moe.moe_attn_decode(q, self.cache, self.table, self.lens, self.q_out, self.ws, sinks=self.sinks)
        self.project(self.q_out.view(B, -1), self.w_o, self.o_x, self.o_w, self.o)
        # residual, and the experts' input
        moe.moe_residual_norm(self.o, self.h, None, None, 1.0, self.h, self.n_mlp, self.mlp_in)
        self.logits = self.mlp_in @ self.w_router.t()
        moe.moe_route_grouped(self.logits, self.sel_bias, k, self.router, self.ids, self.tw, self.ws)
        moe.moe_align_permute(self.ids, E, 16, self.mlp_in, self.sorted, self.offsets, self.blocks, self.row_pos,
                              self.x_perm, self.ws)
        moe.moe_grouped_gemm1_act(self.x_perm, self.sorted, self.offsets, T * k, self.q13, 0,
                                  moe.act(cfg.act, cfg.alpha, cfg.limit), self.act, self.ws)
        moe.moe_grouped_gemm2_weighted(self.act, self.sorted, self.offsets, self.q2, self.tw.view(-1), True, T * k,
                                       self.y, self.ws)
        moe.moe_unpermute_reduce(self.y, self.row_pos, T, k, self.mlp_out, self.ws)
        # the experts' output, normalised, onto the residual
        moe.moe_residual_norm(self.mlp_out, self.h, None, self.n_post, 1.0, self.h, None, None)



def main():
    from bit_block_scaled_gb300 import build
    build.build()
    cfg = get_config("c0")
    block = DecodeBlock(cfg, proj="nvfp4", rope=dict(rot_dim=64, scaling="yarn", base=150000.0, factor=32.0))
    g = torch.Generator().manual_seed(1)
    block.h.copy_(torch.randn(block.B, cfg.H, generator=g))
    block.step()  # loads the kernels
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        block.step()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    n = 31
    start.record()
    for _ in range(n):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    status = moe.moe_read_status(block.ws)
    print(f"{block.B} sequences at {block.lens[0].item()} tokens, {start.elapsed_time(end) / n * 1e3:.1f} us a step, "
          f"status {moe.moe_status_string(status)}, |h| = {block.h.norm().item():.3f}")
    if status:
        raise SystemExit(1)


if __name__ == "__main__":
    main()
