"""How the batch plan, rotary positions and quantisation are launched, over a CUDA runtime that launches nothing
(fake_cuda.py): grids by sizes, kernels by alignment, limits set on each device."""
import pytest

import bit_block_scaled_gb300 as moe
from fake_cuda import Library, link

P = 1 << 20  # stands for every pointer; nothing is read


@pytest.fixture(scope="module")
def path(tmp_path_factory):
    return link(tmp_path_factory.mktemp("fake"))


@pytest.fixture
def lib(path, tmp_path):
    return Library(path, tmp_path)


def plan(lib, B, T, rows_each=0):
    return lib.lib.moe_batch_plan(P, P, B, 16, 1000, P, 100, 100, P, P, P, P, P, T, rows_each, P, P, P, P, None)


def test_plan_clusters(lib):
    for B, T, block, cluster in [(1, 1, 128, 1), (64, 64, 128, 1), (300, 300, 512, 1), (4096, 0, 1024, 1), (8, 2000, 1024, 2),
                                 (8, 5000, 1024, 8), (8, 65536, 1024, 16), (8, 1 << 28, 1024, 16)]:
        assert plan(lib, B, T) == 0
        (name, device, grid, threads, c), = lib.launches()
        assert "plan_kernel" in name and grid[0] == c == cluster and threads == block and device == 0


def test_plan_on_every_device(lib):
    """4096 sequences take as much shared memory as is there without being asked for, and more: asked for on each device."""
    for d in (0, 1, 0):
        lib.device(d)
        assert plan(lib, 4096, 4096) == 0
        assert [l[1] for l in lib.launches()] == [d]


def test_a_limit_that_is_refused_is_asked_for_again(lib):
    lib.lib.fake_refuse(1)
    assert plan(lib, 4, 4) == 3 and not lib.launches()
    assert plan(lib, 4, 4) == 0 and len(lib.launches()) == 1


def rope_struct(rot=64, layout=0):
    return moe.Rope(rot, layout, 1.0, P)


def rope(lib, T, heads, D=64, rot=64, q=P, stride=None):
    st = heads * D if stride is None else stride
    return lib.lib.moe_rope(rope_struct(rot), P, T, D, q, st, D, heads, P + (1 << 30), heads * D, D, None, 0, 0, 0, None, 0, 0, 0, None)


def test_rope_grids(lib):
    for T, heads, grid in [(1, 72, 2), (1, 8, 1), (700, 8, 350), (8192, 40, 2048)]:
        assert rope(lib, T, heads) == 0
        (name, _, g, threads, _), = lib.launches()
        assert "rope_kernel" in name and g[0] == grid and threads == 256, (T, heads, g)


def test_rope_kernels_by_alignment(lib):
    names = []
    for kw in (dict(), dict(q=P + 2), dict(stride=516), dict(rot=40), dict(rot=48)):
        assert rope(lib, 10, 8, **kw) == 0
        names.append(lib.launches()[0][0])
    pieces, pairs, columns = names[0], names[1], names[3]
    assert len({pieces, pairs, columns}) == 3 and names[2] == pairs and names[4] == pieces


def test_rope_write_grid(lib):
    def cache(D):
        return moe.KvCache(2, 1000, 16, 8, D, P)
    for T, q, D, grid in [(64, None, 64, 16), (64, P, 64, 80), (1, P, 128, 2), (12345, None, 128, 1544)]:
        st = 32 * D
        assert lib.lib.moe_rope_kv_write(rope_struct(), P, q, st, D, 32, q, st, D, P, 8 * D, D, P, 8 * D, D, 0, P, T, cache(D), P, None) == 0
        (name, _, g, _, _), = lib.launches()
        assert "rope_write_kernel" in name and g[0] == grid, (T, D, g)


def test_quantize_grids(lib):
    for T, K, grid in [(1, 2880, 1), (64, 2880, 64), (608, 512, 76), (609, 512, 77), (8192, 2880, 2048), (8192, 4096, 2048), (700, 16384, 700)]:
        f = moe.Fp4(0, T, K, 1, P, P, P)
        assert lib.lib.moe_fp4_quantize(P, 0, K, f, None) == 0
        (name, _, g, threads, _), = lib.launches()
        assert "fp4_quantize_kernel" in name and g[0] == grid and threads == 256, (T, K, g)


def test_product_without_an_encoder(lib):
    """No driver, no tensor maps: an error, and nothing launched."""
    f = moe.Fp4(0, 4, 64, 1, P, P, P)
    assert lib.lib.moe_fp4_linear(f, f, None, P, 0, 8, P, None) == 3 and not lib.launches()
