"""Builds libmoe4.so (the C-ABI library) in-tree with nvcc for sm_103a.

Each .cu file is compiled to an object in parallel, then linked into a shared
library next to this file. cudart is linked statically, so the library has no
dependency beyond the CUDA driver. Beside it stands _binding.so, the C++ part of
the Python binding (csrc/binding.cpp), which is built with g++ (or $CXX) against
the installed PyTorch; without a PyTorch with CUDA or a C++ compiler the library
is built alone.
"""
import concurrent.futures as cf
import os
import shlex
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmoe4.so")
BINDING = os.path.join(HERE, "_binding.so")
SOURCES = ["api.cu", "route.cu", "align.cu", "gemm.cu", "unpermute.cu", "static_ws.cu", "convert.cu",
           "block_api.cu", "group_route.cu", "norm.cu", "kvcache.cu", "attn.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _binding_command():
    """The binding's object, the command that compiles it and the one that links it; None without what they need.
    Its ABI is that of the interpreter and the PyTorch it is compiled against (_made_for)."""
    cxx = shlex.split(os.environ.get("CXX") or shutil.which("g++") or "")
    try:
        import torch
    except ImportError:
        return None
    if not cxx or torch.version.cuda is None:
        return None
    top = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    obj = os.path.join(BUILD, "binding.o")
    inc = [os.path.join(top, "include"), os.path.join(top, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    compile_ = [*cxx, "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
                *(x for i in inc for x in ("-isystem", i)), "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
    lib = os.path.join(top, "lib")
    link = [*cxx, "-shared", "-o", BINDING + ".tmp", obj, LIB, "-Wl,-rpath,$ORIGIN", f"-L{lib}",
            f"-Wl,-rpath,{lib}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    return obj, compile_, link


def _made_for(commands):
    """What the binding is made for; one that was made for something else is made anew."""
    import torch
    return "\n".join([str(torch.__version__), str(torch.version.git_version), sys.version, *map(" ".join, commands)])


def _stale(obj, deps):
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose: bool = False, force: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, h) for h in os.listdir(CSRC) if h.endswith((".h", ".cuh"))]
    headers.append(os.path.join(HERE, "..", "include", "moe4.h"))
    cc = nvcc()
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + headers):
            jobs.append([cc, *ARCH, *FLAGS, *extra_flags, "-c", s, "-o", o])

    binding = _binding_command()
    lib_jobs = len(jobs)
    if binding:
        made_for, made_for_path = _made_for(binding[1:]), binding[0] + ".for"
        if os.path.exists(made_for_path):
            with open(made_for_path) as f:
                same = f.read() == made_for
        else:
            same = False
        if force or not same or _stale(binding[0], [os.path.join(CSRC, "binding.cpp"), headers[-1]]):
            jobs.append(binding[1])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    def checked(cmd, r, what):
        if verbose or r.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"{what} failed")

    with cf.ThreadPoolExecutor(max_workers=len(jobs) or 1) as ex:
        done = list(ex.map(run, jobs))
    # the library first, whatever becomes of the binding
    for cmd, r in done[:lib_jobs]:
        checked(cmd, r, f"compiling {cmd[-3]}")
    if force or lib_jobs or not os.path.exists(LIB):
        cmd = [cc, *ARCH, "-shared", "-Xlinker", "-soname=libmoe4.so", "-o", LIB + ".tmp", *objs]
        checked(*run(cmd), "linking the library")
        os.replace(LIB + ".tmp", LIB)
    for cmd, r in done[lib_jobs:]:
        checked(cmd, r, f"compiling {cmd[-3]}")
    if binding and (force or jobs or not os.path.exists(BINDING)):
        checked(*run(binding[2]), "linking the binding")
        os.replace(BINDING + ".tmp", BINDING)
        with open(made_for_path, "w") as f:
            f.write(made_for)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
