"""What the calls around the layer keep between launches is a device's own: a process may use them on several. Two
devices of a stand-in for the CUDA runtime, 152 and 100 SMs."""
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
