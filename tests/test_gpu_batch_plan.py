"""moe_batch_plan against the oracle, value for value: sizes, shortages, ended sequences, bad inputs, in place, captured."""
import numpy as np
import pytest
import torch

import bit_block_scaled_gb300 as moe
from gpu_helpers import built, ws_status
from oracle import plan as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    return built()


def dev(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda").contiguous()


def status_bits(ws):
    word = int(ws[:4].cpu().view(torch.int32)[0])
    return (P.CAPACITY if word & (1 << 7) else 0) + (P.BAD_INDEX if word & (1 << 4) else 0), word & ~((1 << 7) | (1 << 4))


def run(new, lens, table, free, count, page, T, in_place=False, bare=False, rows_each=0):
    B = len(lens)
    n, l, f, c = dev(new), dev(lens), dev(free), dev([count])
    t = dev(np.asarray(table).reshape(B, np.asarray(table).size // B))
    wide = torch.full((B, t.shape[1] + 3), 99, dtype=torch.int32, device="cuda")  # rows that are apart
    wide[:, :t.shape[1]] = t
    t = wide[:, :t.shape[1]]
    slots, pos, seqs = (torch.full((T,), 77, dtype=torch.int32, device="cuda") for _ in range(3))
    offs = torch.full((B + 1,), 77, dtype=torch.int32, device="cuda")
    lo, co = (l, c) if in_place else (torch.full_like(l, 77), torch.full_like(c, 77))
    ws = ws_status()
    extra = {} if bare else dict(positions=pos, seq_ids=seqs, offsets=offs)
    moe.moe_batch_plan(n, l, t, f, c, page, slots, lo, co, ws, rows_each=rows_each, **extra)
    errors, other = status_bits(ws)
    assert other == 0 and (wide[:, t.shape[1]:] == 99).all()
    out = dict(slots=slots, lens=lo, count=co, table=t, free=f)
    if not bare:
        out.update(positions=pos, seq_ids=seqs, offsets=offs)
    return {k: v.cpu().numpy() for k, v in out.items()} | {"errors": errors}


def check(new, lens, table, free, count, page, T, **kw):
    got = run(new, lens, table, free, count, page, T, **kw)
    ref = P.batch_plan(new, lens, np.asarray(table).reshape(len(lens), np.asarray(table).size // len(lens)), free, count, page, T,
                       kw.get("rows_each", 0))
    for k, v in got.items():
        np.testing.assert_array_equal(v.reshape(-1) if k == "count" else v, ref[k], err_msg=k)
    return ref


def state(B, cols, page, seed, new_most=1, ends=0.0, idle=0.0, spare=None):
    """Lengths, a table of distinct pages and a stack of the rest."""
    r = np.random.default_rng(seed)
    lens = np.floor((cols * page + 1) ** r.random(B)).astype(int) - 1
    new = r.integers(1, new_most + 1, B)
    new[r.random(B) < idle] = 0
    new[r.random(B) < ends] = -1
    held = -(-lens // page)
    total = int(held.sum()) + (B * cols if spare is None else spare)
    order = r.permutation(max(total, 1))
    table, at = np.full((B, cols), -1), 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    free = np.full(len(order), -1)
    free[:len(order) - at] = order[at:]
    return new, lens, table, free, len(order) - at


@pytest.mark.parametrize("B,cols,page", [(1, 1, 16), (2, 5, 16), (31, 40, 32), (64, 100, 16), (500, 20, 48), (1024, 3, 64),
                                         (1025, 7, 16), (4096, 4, 128)])
def test_decode(B, cols, page):
    check(*state(B, cols, page, B), page, B)


@pytest.mark.parametrize("B,cols,page,most,T", [(1, 300, 16, 4000, 5000), (7, 64, 32, 500, 2500), (100, 50, 16, 300, 17000),
                                               (1500, 30, 16, 60, 50000), (4096, 9, 16, 40, 100000)])
@pytest.mark.parametrize("ends", [0.0, 0.3])
def test_mixed(B, cols, page, most, T, ends):
    check(*state(B, cols, page, B, most, ends, 0.2), page, T)


@pytest.mark.parametrize("seed", range(6))
def test_shortages(seed):
    """Too few pages, rows or columns: all of a sequence or nothing, in order."""
    B, cols, page = 200, 12, 16
    s = state(B, cols, page, seed, 100, 0.1 * (seed % 3), 0.1, spare=[0, 1, 50, 200, 400, 90][seed])
    ref = check(*s, page, [20000, 3000, 20000, 5000, 100, 1][seed])
    assert ref["errors"] == P.CAPACITY


@pytest.mark.parametrize("B,cols,page,most,rows_each,T", [
    (1, 3, 16, 1, 1, 1), (64, 20, 16, 1, 1, 64), (700, 12, 48, 1, 1, 700), (90, 20, 16, 4, 4, 360), (90, 20, 16, 6, 4, 350),
    (1025, 9, 16, 3, 3, 3075), (4096, 5, 16, 7, 7, 28672), (3, 40, 32, 500, 600, 1700), (5, 9, 16, 1, 1 << 28, 9)])
def test_fixed_rows(B, cols, page, most, rows_each, T):
    """Sequence b keeps its rows, whatever the others do."""
    s = state(B, cols, page, B + most, most, 0.2, 0.2)
    check(*s, page, T, rows_each=rows_each)
    check(*state(B, cols, page, B, most, 0.1, 0.1, spare=B // 8), page, T, rows_each=rows_each, in_place=True)


def test_in_place_and_without_the_rest():
    s = state(300, 30, 32, 5, 90, 0.2, 0.1)
    check(*s, 32, 20000, in_place=True)
    check(*s, 32, 20000, bare=True)


def test_empty_batches():
    ws = ws_status()
    none, one = torch.zeros(0, dtype=torch.int32, device="cuda"), dev([3])
    slots = torch.full((5,), 77, dtype=torch.int32, device="cuda")
    offs = torch.full((1,), 77, dtype=torch.int32, device="cuda")
    moe.moe_batch_plan(none, none, torch.zeros(0, 4, dtype=torch.int32, device="cuda"), dev([0, 1, 2, 3]), one, 16, slots, none,
                       one, ws, offsets=offs)
    assert (slots == -1).all() and one.item() == 3 and offs.item() == 0
    check([0, 0], [5, 16], [[0], [1]], [2, -1, -1], 1, 16, 0)
    check([1, 2], [0, 0], np.zeros((2, 0)), [0], 1, 16, 4)  # a table without columns


def test_bad_inputs():
    table = [[0, 1], [2, 3], [4, 5]]
    for lens in ([-1, 5, 20], [33, 5, 20], [2 ** 31 - 1, -2 ** 31, 1]):
        ref = check([1, 1, 1], lens, table, [6, 7, 8, 9, 1, 1, 1, 1, 1, 1], 4, 16, 3)
        assert ref["errors"] & P.BAD_INDEX
    for count in (-1, 11, 2 ** 31 - 1, -2 ** 31):
        check([1, 20, 1], [16, 5, 31], table, [6, 7, 8, 9, 1, 1, 1, 1, 1, 1], count, 16, 30)
    # pages that are none, on the stack and in the table
    check([17, 1, 1], [0, 5, 20], [[-1, -1], [-7, 3], [4, 99]], [6, 100, -3, 9], 4, 16, 30)
    # more pages come back than there are
    check([-1, -1, 3], [32, 32, 0], [[0, 1], [2, 3], [-1, -1]], [0, 1, 2, 3], 3, 16, 4)
    # tokens past 31 bits
    big = 2 ** 31 - 1
    check([big, big, 1], [0, 0, 0], table, [6, 7, 8, 9], 4, 16, 8)


def test_steps_of_a_captured_plan():
    """In place in a graph: sequences grow token by token, as one call by the oracle after another."""
    B, cols, page = 40, 6, 16
    new, lens, table, free, count = state(B, cols, page, 3)
    lens = np.minimum(lens, 40)
    n, l, t, f, c = dev(np.ones(B)), dev(lens), dev(table), dev(free), dev([count])
    slots, pos, ws = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda"), ws_status()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_batch_plan(n, l, t, f, c, page, slots, l, c, ws, positions=pos)
    for _ in range(20):
        ref = P.batch_plan(np.ones(B), lens, table, free, count, page, B)
        g.replay()
        for got, k in ((slots, "slots"), (pos, "positions"), (l, "lens"), (t, "table"), (f, "free"), (c, "count")):
            np.testing.assert_array_equal(got.cpu().numpy().reshape(np.shape(ref[k]) or (1,)), ref[k], err_msg=k)
        lens, table, free, count = ref["lens"], ref["table"], ref["free"], ref["count"]
    assert status_bits(ws) == (0, 0)
