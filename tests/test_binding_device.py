"""The binding launches on its tensors' device, whichever is current: its object over a CUDA runtime that launches
nothing, with tensors on two devices that are none."""
import ctypes
import importlib.machinery
import importlib.util
import os
import subprocess

import pytest
import torch

import bit_block_scaled_gb300 as moe
import fake_cuda
from bit_block_scaled_gb300 import build as B

bf16, i32 = torch.bfloat16, torch.int32


def load(name, path):
    loader = importlib.machinery.ExtensionFileLoader(name, path)
    mod = importlib.util.module_from_spec(importlib.util.spec_from_loader(name, loader))
    loader.exec_module(mod)
    return mod


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    """(binding, device module, library)"""
    where = tmp_path_factory.mktemp("binding")
    lib = fake_cuda.link(where)
    obj, compile_, link = B._binding_command()
    binding = os.path.join(where, "_binding.so")
    subprocess.run([lib if a == B.LIB else binding if a == B.BINDING + ".tmp" else a for a in link], check=True)
    device, dev_obj = os.path.join(where, "_fake_device.so"), os.path.join(where, "fake_device.o")
    src = os.path.join(fake_cuda.HERE, "fake_device.cpp")
    subprocess.run([{os.path.join(B.CSRC, "binding.cpp"): src, obj: dev_obj}.get(a, a) for a in compile_], check=True)
    subprocess.run([{B.LIB: lib, B.BINDING + ".tmp": device, obj: dev_obj}.get(a, a) for a in link], check=True)
    handle = fake_cuda.Library.__new__(fake_cuda.Library)
    handle.lib = ctypes.CDLL(lib)
    handle.lib.fake_launch.restype = ctypes.POINTER(fake_cuda.Launch)
    return load("_binding", binding), load("_fake_device", device), handle


def cache(fmt="fp8", H=2, D=64):
    return moe.KvCache(moe.KV_FMT[fmt], 8, 16, H, D, 1 << 20)


def calls(on):
    """Each call of the binding with its arguments; on(tensor) puts them on the device."""
    x = on(torch.zeros(4, 64, dtype=bf16))
    kv = on(torch.zeros(3, 2, 64, dtype=bf16))
    ws = on(torch.zeros(4096, dtype=torch.uint8))
    big = on(torch.zeros(moe.moe_attn_workspace_size(4, 2, 64), dtype=torch.uint8))
    slots, q = on(torch.zeros(3, dtype=i32)), on(torch.zeros(2, 4, 64, dtype=bf16))
    return {
        "route_grouped": (on(torch.zeros(4, 16)), None, 2, moe.router(), on(torch.zeros(4, 2, dtype=i32)),
                          on(torch.zeros(4, 2)), ws, 0),
        "residual_norm": (x, x, None, None, 1.0, x, None, None, 0),
        "kv_write": (kv, kv, slots, cache(), ws, 0),
        "kv_read": (cache(), slots, kv, None, ws, 0),
        "attn_decode": (q, cache(), on(torch.zeros(2, 2, dtype=i32)), on(torch.zeros(2, dtype=i32)), q, big, 0.1, 0, None,
                        None, 0),
    }


@pytest.mark.parametrize("name", ["route_grouped", "residual_norm", "kv_write", "kv_read", "attn_decode"])
@pytest.mark.parametrize("device", [0, 1])
def test_launches_on_the_tensors_device(fake, name, device):
    binding, mod, lib = fake
    args = calls(lambda t: mod.tensor(device, t))[name]
    lib.launches()
    assert getattr(binding, name)(*args) == 0
    assert [l[1] for l in lib.launches()] == [device]
    assert mod.current() == 0    # what was current is so again


@pytest.mark.parametrize("name", ["route_grouped", "residual_norm", "kv_write", "kv_read", "attn_decode"])
def test_refusals_leave_the_device(fake, name):
    binding, mod, lib = fake
    args = list(calls(lambda t: mod.tensor(1, t))[name])
    last = max(i for i, a in enumerate(args) if isinstance(a, torch.Tensor))
    args[last] = mod.tensor(0, args[last])  # on another device than the rest
    assert getattr(binding, name)(*args) == 1
    assert lib.launches() == [] and mod.current() == 0


@pytest.mark.parametrize("name", ["kv_write", "kv_read", "attn_decode"])
def test_a_cache_in_other_memory_is_refused(fake, name):
    """A cache in host memory (or on another device) would be written and read by a kernel all the same."""
    binding, mod, lib = fake
    args = list(calls(lambda t: mod.tensor(1, t))[name])
    at = next(i for i, a in enumerate(args) if isinstance(a, moe.KvCache))
    host = torch.zeros(8, 2, 1, moe.moe_kv_record_bytes("fp8", 64), dtype=torch.uint8)
    args[at] = moe.kv_cache(host, "fp8", 64)
    assert getattr(binding, name)(*args) == 1 and lib.launches() == []
    args[at] = moe.kv_cache(mod.tensor(1, host), "fp8", 64)
    assert getattr(binding, name)(*args) == 0 and len(lib.launches()) > 0


@pytest.mark.parametrize("part", ["post", "pre"])
def test_a_norms_parameters_in_other_memory_are_refused(fake, part):
    binding, mod, lib = fake
    x, w = mod.tensor(0, torch.zeros(4, 64, dtype=bf16)), torch.ones(64)

    def run(n, x=x):
        post, pre, y = (n, None, None) if part == "post" else (None, n, x)
        return binding.residual_norm(x, x, None, post, 1.0, x, pre, y, 0)
    assert run(moe.norm("rms", mod.tensor(0, w))) == 0 and len(lib.launches()) == 1
    assert run(moe.norm("rms", w)) == 1
    assert run(moe.norm("layer", None, w)) == 1
    # an address that is null, as it is on this device, stands for no weight
    assert run(moe.norm("rms", w.to("meta")), torch.zeros(4, 64, dtype=bf16)) == 1
    assert lib.launches() == []
    with pytest.raises(moe.MoeError):
        moe.norm("layer", w, mod.tensor(0, w))
