"""The calls around the layer over a stand-in for the CUDA runtime with two devices, of 152 and 100 SMs. What they keep
between launches is a device's own: a process may use them on several."""
import threading

import pytest

import fake_cuda

CUDA = 3


@pytest.fixture(scope="module")
def linked(tmp_path_factory):
    return fake_cuda.link(tmp_path_factory.mktemp("fake"))


@pytest.fixture
def lib(linked, tmp_path):
    return fake_cuda.Library(linked, tmp_path)


@pytest.mark.parametrize("fmt", ["bf16", "fp16", "fp8", "nvfp4"])
@pytest.mark.parametrize("D,G", [(64, 4), (64, 16), (128, 4), (128, 16), (256, 8)])
def test_attention_on_a_second_device(lib, fmt, D, G):
    """More than 48 KB of shared memory have to be asked for on each device."""
    for d in (0, 1, 0):
        lib.device(d)
        assert lib.attention(fmt, D, G=G) == 0
    assert [l[1] for l in lib.launches()] == [0, 1, 0]


def test_grids_follow_the_device(lib):
    for d, sms in enumerate(fake_cuda.SMS):
        lib.device(d)
        assert lib.attention(B=8, H=8, pages=5000) == 0
        assert lib.launches()[0][2][0] == min(4 * sms, 640)
        assert lib.route(100000) == 0
        assert lib.launches()[0][2][0] == 4 * sms
        assert lib.norm(5000, 2880) == 0
        assert lib.launches()[0][2][0] % sms == 0
        # a CTA a row up to two rows an SM
        assert lib.norm(250, 2880) == 0
        assert ("norm_walk" in lib.launches()[0][0]) == (250 > 2 * sms)


def test_a_failure_is_not_kept(lib):
    lib.lib.fake_refuse(1)
    assert lib.attention() == CUDA and lib.launches() == []
    assert lib.attention() == 0


def test_first_calls_of_several_threads(lib):
    codes = []
    go = threading.Barrier(8)

    def first():
        go.wait()
        codes.append(lib.attention("fp8", 128))
    threads = [threading.Thread(target=first) for _ in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert codes == [0] * 8 and all(l[2][0] > 0 for l in lib.launches())


@pytest.mark.parametrize("T,H,t,h", [(3, 3, 192, 64), (3, 3, 64, 192), (3, 3, 200, 64), (3, 3, 64, 256), (1, 3, 0, 64), (1, 3, 0, 72), (3, 1, 64, 0), (1, 1, 0, 0), (2, 3, 64, 128), (3, 2, 128, 64), (2, 1, 1 << 40, 0),
                                     (2, 3, 1 << 40, 64), (2, 3, 64, 1 << 40),
                                     (3, 3, 128, 192), (3, 3, 192, 128)])
def test_outputs_whose_rows_lie_apart_are_taken(lib, T, H, t, h):
    """Tokens or heads outermost, spaces between them, strides of dimensions of one."""
    P = 1 << 20
    c = fake_cuda.moe.KvCache(2, 8, 16, H, 64, P)
    assert lib.lib.moe_kv_read(c, P, T, P, None, 0, t, h, 0, 0, P, None) == 0
    assert lib.lib.moe_kv_read(c, P, T, None, P, 0, 0, 0, t, h, P, None) == 0
    assert lib.lib.moe_attn_decode(P, 0, H * 64, 64, c, P, 2, 2, P, T, H, 0.1, 0, None, P, t, h, None, P, 1 << 30, None) == 0
    assert len(lib.launches()) == 3
    assert lib.lib.moe_kv_read(c, P, 3, P, None, 0, 1 << 60, 1 << 60, 0, 0, P, None) == (1 if H > 1 else 0)
