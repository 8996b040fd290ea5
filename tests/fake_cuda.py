"""The library's host code over a CUDA runtime that launches nothing (fake_cudart.c): argument checks, the choice of
kernels and grids, and what is kept for each device, without a GPU."""
import ctypes
import glob
import os
import shutil
import subprocess

import bit_block_scaled_gb300 as moe
from bit_block_scaled_gb300 import build as B

HERE = os.path.dirname(os.path.abspath(__file__))
SMS = (152, 100)


class Launch(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char_p), ("device", ctypes.c_int), ("grid", ctypes.c_uint * 3),
                ("block", ctypes.c_uint), ("smem", ctypes.c_uint), ("cluster", ctypes.c_uint)]


def link(where):
    """The library's objects and the runtime's stand-in, in one shared object; its path."""
    B.build()
    path = os.path.join(str(where), "fake.so")
    objs = [os.path.join(B.BUILD, s.replace(".cu", ".o")) for s in B.SOURCES]
    fake = os.path.join(str(where), "fake_cudart.o")
    subprocess.run(["gcc", "-O1", "-fPIC", "-c", os.path.join(HERE, "fake_cudart.c"), "-o", fake], check=True)
    subprocess.run(["g++", "-shared", "-Wl,-Bsymbolic", "-o", path, *objs, fake, "-lpthread", "-ldl"], check=True)
    return path


class Library:
    """A copy of it with nothing kept yet; `device` is the current one."""

    def __init__(self, path, where):
        own = os.path.join(str(where), f"fake{len(glob.glob(os.path.join(str(where), 'fake*.so')))}.so")
        shutil.copy(path, own)
        self.lib = ctypes.CDLL(own)
        for name, (res, args) in moe._lib._SIGS.items():
            f = getattr(self.lib, name)
            f.restype, f.argtypes = res, args
        self.lib.fake_launch.restype = ctypes.POINTER(Launch)

    def device(self, d):
        self.lib.fake_device(d)

    def launches(self):
        out = [self.lib.fake_launch(i).contents for i in range(self.lib.fake_launches())]
        out = [(l.name.decode(), l.device, tuple(l.grid), l.block, l.cluster) for l in out]
        self.lib.fake_clear()
        return out

    def attention(self, fmt="bf16", D=128, H=2, G=4, B=1, pages=100, page=16, window=0):
        P = 1 << 20  # stands for every pointer; nothing is read
        c = moe.KvCache(moe.KV_FMT[fmt], 1000, page, H, D, P)
        q = 1 if fmt == "fp16" else 0
        return self.lib.moe_attn_decode(P, q, H * G * D, D, c, P, pages, pages, P, B, H * G, 0.1, window, None, P, H * G * D, D,
                                        None, P, 1 << 30, None)

    def route(self, T, E=256, k=8):
        P = 1 << 20
        return self.lib.moe_route_grouped(P, 2, E, None, T, E, k, moe.router(), P, P, P, None)

    def norm(self, T, H):
        P = 1 << 20
        n = moe.Norm(0, 2, 1e-5, 0.0, None, None)
        return self.lib.moe_residual_norm(P, H, P, H, None, 0, 0, T, H, 0, 0, n, 1.0, P, H, n, P, H, None)
