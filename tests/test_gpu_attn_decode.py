"""moe_attn_decode against the float64 oracle.

Bounds: a score is a sum of D products in fp32, off by at most ds = D 2^-23 of scale * sum |q||k| (and 2^-22 of its
size for the factors and the base-2 logarithm); a probability by that and 2^-21 for exp2 and the joins, and by half a
step of the type it is multiplied in (bf16 2^-8, f16 2^-11); the output's own rounding is half a step more. So
|out - ref| <= 2 (ds + 2^-20) A + hp A + half |ref| with A = sum p |v|, and |lse - ref| <= ds + 2^-20 (1 + |ref|).
Where p is multiplied as f16, its subnormals have an absolute step: half of 2^-24 where the largest p times its row
scale is 2^11 at least, and the row scale is at most 2 / 448 of a row's largest value times 448 (2688 for both in
NVFP4), so each of n tokens adds at most 2^-35 of the largest p max |v|."""
import numpy as np
import pytest
import torch

import bit_block_scaled_gb300 as moe
from gpu_helpers import built
from oracle import kvcache as KV

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}

#: the smallest positive value of each type
SMALLEST = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}


@pytest.fixture(scope="module", autouse=True)
def lib():
    return built()


def assert_within(got, ref, tol):
    off = ~(np.abs(got - ref) <= tol)
    if off.any():
        i = np.unravel_index(np.argmax(np.where(off, np.abs(got - ref) / tol, 0)), off.shape)
        raise AssertionError(f"{off.sum()} of {off.size} outside, worst at {i}: {got[i]} for {ref[i]}, tol {tol[i]}")


class Case:
    """A cache filled through moe_kv_write, its table and lengths."""

    def __init__(self, lens, H=2, G=4, D=64, fmt="bf16", page=16, q_type=None, seed=0, spare=2, junk=True, kv=None):
        g = torch.Generator().manual_seed(seed)
        self.B, self.H, self.G, self.D, self.fmt, self.page = len(lens), H, G, D, fmt, page
        self.lens = torch.tensor(lens, dtype=torch.int32)
        need = [-(-n // page) for n in lens]
        pages = sum(need) + spare
        order = torch.randperm(pages, generator=g).to(torch.int32)
        self.table = torch.full((self.B, max(need + [1])), -5, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        # whatever lies past a sequence's length must not matter: NaN patterns everywhere first
        self.data = torch.full((pages, H, page // 16, KV.record_bytes(fmt, D)), 0xFF if junk else 0, dtype=torch.uint8,
                               device="cuda")
        self.cache = moe.kv_cache(self.data, fmt, D)
        slots = [int(self.table[b, i // page]) * page + i % page for b, n in enumerate(lens) for i in range(n)]
        T = len(slots)
        k = torch.randn(T, H, D, generator=g) * torch.exp(0.3 * torch.randn(T, H, 1, generator=g))
        v = torch.randn(T, H, D, generator=g) * torch.exp(torch.randn(T, H, 1, generator=g))
        if kv:
            k, v = kv(k, v)
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        if T:
            moe.moe_kv_write(k.cuda(), v.cuda(), torch.tensor(slots, dtype=torch.int32).cuda(), self.cache, ws)
        self.q_type = TYPES[q_type or ("fp16" if fmt == "fp16" else "bf16")]
        self.q = (torch.randn(self.B, H * G, D, generator=g) * 2).to(self.q_type).cuda()
        self.sinks = torch.randn(H * G, generator=g)

    def run(self, scale=None, window=0, sinks=False, lse=True, table=None, lens=None, q=None, out=None, ws=None, stream=None):
        n = moe.moe_attn_workspace_size(self.H * self.G, self.H, self.D)
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda") if ws is None else ws
        out = torch.full(self.q.shape, float("nan"), dtype=self.q_type, device="cuda") if out is None else out
        l = torch.full((self.B, self.H * self.G), float("nan"), device="cuda") if lse else None
        moe.moe_attn_decode(self.q if q is None else q, self.cache, (self.table if table is None else table).cuda(),
                            (self.lens if lens is None else lens).cuda(), out, ws, scale, window,
                            self.sinks.cuda() if sinks else None, l, stream)
        self.status = moe.moe_read_status(ws, stream)
        return out, l

    def check(self, scale=None, window=0, sinks=False, table=None, lens=None, status=0):
        out, lse = self.run(scale, window, sinks, True, table, lens)
        assert self.status == status
        keys, vals = KV.values(self.data.cpu().numpy(), self.fmt, self.D)
        sc = self.D ** -0.5 if scale is None else scale
        ref, rl, mag, size, peak = KV.attend(self.q.double().cpu().numpy(), keys, vals,
                                       (self.table if table is None else table).numpy(),
                                       (self.lens if lens is None else lens).numpy(), sc, window,
                                       self.sinks.double().numpy() if sinks else None)
        o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
        ds = (self.D * 2.0 ** -23 * size + 2.0 ** -22 * size)
        hp = 2.0 ** -8 if self.fmt == "bf16" else 2.0 ** -11
        half = torch.finfo(self.q_type).eps / 2
        tiny = SMALLEST[self.q_type] / 2
        tol = (2 * (ds[:, :, None] + 2.0 ** -20) + hp) * (1 + half) * mag + half * np.abs(ref) + tiny
        if self.fmt != "bf16":
            tol += 2.0 ** -35 * peak[:, :, None]
        assert_within(o, ref, tol)
        live = np.isfinite(rl)
        assert np.array_equal(l[~live], rl[~live])
        assert_within(l[live], rl[live], (ds + 2.0 ** -20 * (1 + np.abs(rl)))[live])
        return out, lse


FMTS = ["bf16", "fp16", "fp8", "nvfp4"]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 130])
def test_lengths(fmt, D, n):
    Case([n], H=1, G=8, D=D, fmt=fmt).check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("G", [1, 3, 5, 8, 9, 16, 17, 40])
def test_heads_of_a_group(fmt, G):
    Case([70, 5], H=2, G=G, D=64, fmt=fmt).check(sinks=True)
    Case([33], H=1, G=G, D=256, fmt=fmt).check()
    Case([33], H=1, G=G, D=128, fmt=fmt).check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page", [16, 48, 64, 256])
def test_ragged_batches_and_pages(fmt, page):
    Case([300, 0, 1, 17, 257, 64, 0, 999, 16], H=3, G=4, D=64, fmt=fmt, page=page).check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 128, 5000])
def test_windows(fmt, window):
    c = Case([300, 0, 1, 90, 128, 129], H=2, G=5, D=64, fmt=fmt, page=32)
    c.check(window=window)
    c.check(window=window, sinks=True)


@pytest.mark.parametrize("fmt", FMTS)
def test_split_over_many_blocks(fmt):
    """Long enough that every (sequence, head) falls to many CTAs, and short ones lie between."""
    Case([5000, 3, 2900], H=2, G=8, D=64, fmt=fmt, page=64).check(sinks=True)
    Case([9000], H=1, G=2, D=128, fmt=fmt, page=16).check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lens,H", [
    ([600, 0, 1, 40, 520], 3),                  # clusters of 8
    ([300, 5, 0, 259], 8),                      # of 4
    ([130, 129, 0, 17, 90] * 4, 6),             # of 2
    ([100, 0, 64, 1] * 10, 5),                  # single CTAs
    ([33, 0, 128, 64, 7, 90, 15, 1] * 25, 4),   # whole ones, several a CTA
    ([1100, 0, 3, 1090] * 3, 40),               # even shares
])
def test_ways_of_sharing_the_work(fmt, lens, H):
    c = Case(lens, H=H, G=2, D=64, fmt=fmt, page=16)
    c.check(sinks=True)
    if len(lens) < 8:
        c.check(window=100)
        t = c.table.clone()
        t[0, 1] = -1
        c.check(table=t, status=5)


def test_many_short_sequences():
    rng = np.random.default_rng(0)
    Case(rng.integers(0, 40, size=700).tolist(), H=2, G=2, D=64, fmt="fp8").check()


def test_empty_rows():
    c = Case([0, 0], H=1, G=2)
    out, lse = c.check()
    assert not out.any() and torch.all(lse == -float("inf"))
    out, lse = c.check(sinks=True)
    assert not out.any() and torch.allclose(lse.cpu(), c.sinks.expand(2, 2))


@pytest.mark.parametrize("fmt", FMTS)
def test_large_and_peaked_scores(fmt):
    c = Case([500], H=1, G=4, D=64, fmt=fmt)
    c.check(scale=4.0)
    c.check(scale=-1.0)
    c.check(scale=0.0)
    c.sinks[:] = torch.tensor([80.0, -80.0, 0.0, -float("inf")])
    c.check(sinks=True)


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
def test_rows_of_very_different_sizes(fmt):
    """One value far larger than the others under a vanishing probability, rows of zeros, tiny rows: probabilities
    are held relative to what they weigh, so the small rows keep their precision."""
    def kv(k, v):
        k[0] *= 0.0
        v[0] *= 2.0 ** 20
        k[1:] += 1.0
        v[5::7] = 0.0
        v[6::7] *= 2.0 ** -30
        return k, v
    for s in range(3):
        c = Case([200], H=1, G=4, D=64, fmt=fmt, kv=kv, seed=s)
        c.q = c.q.abs() + 3.0
        c.check()
    Case([40], H=1, G=4, D=64, fmt=fmt, kv=lambda k, v: (k, v * 0.0)).check()


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("q_type", ["bf16", "fp16"])
def test_query_types_and_sizes(fmt, q_type):
    c = Case([100], H=1, G=3, D=128, fmt=fmt, q_type=q_type)
    c.check()
    c.q[0, 0] *= 0.0
    c.q[0, 1] *= 2.0 ** -10
    c.check()
    if q_type == "bf16":
        c.q[0, 2] = c.q[0, 2] * 2.0 ** 60
        c.check(scale=2.0 ** -62)


@pytest.mark.parametrize("fmt", FMTS)
def test_nan_in_a_key_or_value(fmt):
    """A NaN that is read comes out; where it comes from a value, only in its column for 16-bit caches."""
    def kv(k, v):
        k[3, 0, 7] = float("nan")
        v[9, 1, 5] = float("nan")
        return k, v
    c = Case([30], H=3, G=2, D=64, fmt=fmt, kv=kv)
    out, lse = c.run()
    assert torch.isnan(out[0, :2]).all() and torch.isnan(lse[0, :2]).all()
    assert torch.isnan(out[0, 2:4, 5]).all() and torch.isfinite(lse[0, 2:]).all()
    if fmt in ("bf16", "fp16"):
        assert torch.isfinite(out[0, 2:4, :5]).all()
    else:
        assert torch.isnan(out[0, 2:4]).all()
    assert torch.isfinite(out[0, 4:]).all()
    out, _ = c.run(window=20)     # tokens 10..29: neither is read
    assert torch.isfinite(out).all()
    long = Case([3000], H=3, G=2, D=64, fmt=fmt, kv=kv)   # split over blocks and joined
    out, lse = long.run()
    assert torch.isnan(out[0, :2]).all() and torch.isnan(lse[0, :2]).all() and torch.isnan(out[0, 2:4, 5]).all()
    assert torch.isfinite(out[0, 4:]).all() and torch.isfinite(lse[0, 2:]).all()


def test_bad_pages_and_lengths():
    c = Case([100, 60], H=2, G=2)
    t = c.table.clone()
    t[0, 2], t[1, 0] = 1 << 20, -1
    c.check(table=t, status=5)
    c.check(lens=torch.tensor([100, -3], dtype=torch.int32), status=5)
    c = Case([112, 112], H=2, G=2)
    c.check(lens=torch.tensor([112, 113], dtype=torch.int32), status=5)


def test_strided_query_and_output():
    c = Case([300, 40], H=2, G=4, D=64, fmt="nvfp4")
    want, _ = c.run()
    wide = torch.zeros(2, 24, 64, dtype=c.q_type, device="cuda")
    wide[:, 8:16] = c.q
    out = torch.zeros(8, 2, 2, 64, dtype=c.q_type, device="cuda")
    o = out[:, :, 1].transpose(0, 1)
    c.run(q=wide[:, 8:16], out=o)
    assert torch.equal(o, want) and not out[:, :, 0].any()
    table = torch.full((2, 50), -1, dtype=torch.int32)
    table[:, 7:7 + c.table.shape[1]] = c.table
    got, _ = c.run(table=table[:, 7:7 + c.table.shape[1]])
    assert torch.equal(got, want)


@pytest.mark.parametrize("fmt", ["bf16", "nvfp4"])
def test_repeats_are_identical_with_a_used_workspace(fmt):
    c = Case([2000, 31, 700], H=2, G=8, D=128, fmt=fmt)
    want, wl = c.run(sinks=True)
    ws = torch.randint(0, 256, (moe.moe_attn_workspace_size(16, 2, 128),), dtype=torch.uint8, device="cuda")
    moe.moe_clear_status(ws)
    for _ in range(3):
        got, gl = c.run(sinks=True, ws=ws)
        assert torch.equal(got, want) and torch.equal(gl, wl) and c.status == 0


def test_graph_and_stream():
    """Captured once, replayed after more tokens were written: lengths are read on the device."""
    c = Case([400, 90], H=2, G=4, D=64, fmt="fp8", page=64)
    ws = torch.zeros(moe.moe_attn_workspace_size(8, 2, 64), dtype=torch.uint8, device="cuda")
    out, lens, table = torch.zeros_like(c.q), c.lens.cuda() - 50, c.table.cuda()
    moe.moe_attn_decode(c.q, c.cache, table, lens, out, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        moe.moe_attn_decode(c.q, c.cache, table, lens, out, ws)
    lens.copy_(c.lens)
    graph.replay()
    torch.cuda.synchronize()
    want, _ = c.run()
    assert torch.equal(out, want)


def test_a_cache_past_four_gigabytes():
    D, H, page, pages = 128, 8, 128, 20000
    data = torch.zeros(pages, H, page // 16, KV.record_bytes("bf16", D), dtype=torch.uint8, device="cuda")
    cache = moe.kv_cache(data, "bf16", D)
    g = torch.Generator().manual_seed(0)
    k, v = (torch.randn(page, H, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    ws = torch.zeros(moe.moe_attn_workspace_size(H, H, D), dtype=torch.uint8, device="cuda")
    last = (pages - 1) * page + torch.arange(page, dtype=torch.int32, device="cuda")
    moe.moe_kv_write(k, v, last, cache, ws)
    q = torch.randn(1, H, D, generator=g).to(torch.bfloat16).cuda()
    out = torch.empty_like(q)
    moe.moe_attn_decode(q, cache, torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda"),
                        torch.tensor([page], dtype=torch.int32, device="cuda"), out, ws)
    p = torch.softmax(torch.einsum("hd,nhd->hn", q[0].double(), k.double()) * D ** -0.5, 1)
    ref = torch.einsum("hn,nhd->hd", p, v.double())
    mag = torch.einsum("hn,nhd->hd", p, v.double().abs())
    assert torch.all((out[0].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -7 * mag)


def wide(c, columns, page=-5):
    """The case's table as a program holds it whose contexts may grow to `columns` pages."""
    t = torch.full((c.B, columns), page, dtype=torch.int32)
    t[:, :c.table.shape[1]] = c.table
    return t


def is_split(c, **kw):
    """Checks the case, which has to go through the workspace and the second kernel."""
    c.check(**kw)
    assert moe.moe_last_launch_count() == 2


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,G", [(64, 1), (64, 9), (64, 16), (64, 17), (64, 40), (128, 8), (128, 9), (128, 40), (256, 8),
                                 (256, 12)])
def test_partials_of_every_shape(fmt, D, G):
    """Two column tiles a CTA, several blocks of heads, the widest heads: split over CTAs and joined."""
    c = Case([4700, 3, 0, 777], H=2, G=G, D=D, fmt=fmt, page=32)
    is_split(c, sinks=True)
    is_split(c, window=4500)
    t = c.table.clone()
    t[0, 5], t[0, 60:100], t[3, 0] = -1, 1 << 20, c.data.shape[0]
    is_split(c, table=t, status=5)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lens,H", [([600, 0, 1, 40, 520], 3), ([130, 129, 0, 17, 90] * 4, 6),
                                    ([33, 0, 128, 64, 7, 90, 15, 1] * 25, 4), ([1100, 0, 3, 1090] * 3, 40), ([1], 1)])
def test_tables_wider_than_the_lengths(fmt, lens, H):
    c = Case(lens, H=H, G=2, D=64, fmt=fmt, page=16)
    is_split(c, table=wide(c, 4096), sinks=True)
    if len(lens) < 8:
        c.check(table=wide(c, 4096), window=100)


@pytest.mark.parametrize("fmt", FMTS)
def test_nan_through_the_join(fmt):
    """In one CTA's share of a sequence that many have; other heads and, with 16-bit caches, other columns are clear."""
    def kv(k, v):
        k[4003, 0, 7] = float("nan")
        v[2009, 1, 5] = float("nan")
        return k, v
    c = Case([6000], H=3, G=2, D=64, fmt=fmt, kv=kv)
    out, lse = c.run(sinks=True)
    assert moe.moe_last_launch_count() == 2
    assert torch.isnan(out[0, :2]).all() and torch.isnan(lse[0, :2]).all()
    assert torch.isnan(out[0, 2:4, 5]).all() and torch.isfinite(lse[0, 2:]).all()
    if fmt in ("bf16", "fp16"):
        assert torch.isfinite(out[0, 2:4, 6:]).all()
    assert torch.isfinite(out[0, 4:]).all()


@pytest.mark.parametrize("fmt,D,G", [("bf16", 128, 8), ("nvfp4", 64, 16), ("fp8", 256, 12)])
def test_split_repeats_are_identical_with_a_used_workspace(fmt, D, G):
    c = Case([6000, 31, 700], H=2, G=G, D=D, fmt=fmt)
    want, wl = c.run(sinks=True)
    assert moe.moe_last_launch_count() == 2
    for fill in (0xFF, 0x7F, 0x00):
        ws = torch.full((moe.moe_attn_workspace_size(2 * G, 2, D),), fill, dtype=torch.uint8, device="cuda")
        moe.moe_clear_status(ws)
        for _ in range(2):
            got, gl = c.run(sinks=True, ws=ws)
            assert torch.equal(got, want) and torch.equal(gl, wl) and c.status == 0


def test_split_in_a_graph_with_growing_lengths():
    c = Case([5200, 90], H=2, G=4, D=64, fmt="fp8", page=64)
    ws = torch.zeros(moe.moe_attn_workspace_size(8, 2, 64), dtype=torch.uint8, device="cuda")
    out, lens, table = torch.zeros_like(c.q), torch.zeros_like(c.lens).cuda(), c.table.cuda()
    moe.moe_attn_decode(c.q, c.cache, table, lens, out, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        moe.moe_attn_decode(c.q, c.cache, table, lens, out, ws)
    assert moe.moe_last_launch_count() == 2
    for less in (5000, 17, 0):
        lens.copy_((c.lens - less).clamp(min=0))
        graph.replay()
        torch.cuda.synchronize()
        want, _ = c.run(lens=lens.cpu())
        assert torch.equal(out, want)
