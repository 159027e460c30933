"""Build libpa.so (CUDA kernels + C ABI + host block pool) for sm_100a, and
_binding, the Python extension in front of it (csrc/binding.cpp).

Usage: ``python -m paged_kv_cache_429_b200.build`` (or via
``__graft_entry__.build()``). The library is written next to this file so it
travels with the source tree. ``--library`` builds libpa.so alone, for callers
of the C ABI: the extension also needs Python's and torch's headers.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libpa.so")

SOURCES = [os.path.join(CSRC, "pa_api.cu"), os.path.join(CSRC, "pa_noalloc.cu"),
           os.path.join(CSRC, "pool.cpp")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in os.listdir(CSRC)
                  if f.endswith((".cuh", ".h"))] + [os.path.join(INCLUDE, "pa.h")]

BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(HERE, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
BINDING_DEPS = [BINDING_SOURCE, os.path.join(INCLUDE, "pa.h")]
BINDING_STAMP = os.path.join(HERE, "_build", "binding.txt")  # the torch it was built with

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-shared",
]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _newer(target: str, deps) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(f) <= t for f in deps)


def up_to_date() -> bool:
    return _newer(LIB, DEPS)


def _torch_id() -> str:
    import torch
    return f"torch {torch.__version__} abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)}\n"


def binding_up_to_date() -> bool:
    """Newer than its sources, and built with the torch that is here now."""
    if not _newer(BINDING, BINDING_DEPS) or not os.path.exists(BINDING_STAMP):
        return False
    with open(BINDING_STAMP) as f:
        return f.read() == _torch_id()


def build_binding(force: bool = False) -> str:
    """The extension links libpa.so next to it, and the torch it is run with."""
    if not force and binding_up_to_date():
        return BINDING
    import torch
    troot = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    include = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(troot, "include"),
               os.path.join(troot, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    for d in include:
        cmd += ["-isystem" if d is not INCLUDE else "-I", d]
    cmd += ["-o", BINDING, BINDING_SOURCE, "-L", HERE, "-lpa", "-L", os.path.join(troot, "lib"),
            "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    if os.path.exists(BINDING_STAMP):
        os.remove(BINDING_STAMP)
    subprocess.run(cmd, check=True)
    os.makedirs(os.path.dirname(BINDING_STAMP), exist_ok=True)
    with open(BINDING_STAMP, "w") as f:
        f.write(_torch_id())
    return BINDING


def build(force: bool = False, verbose: bool = False, binding: bool = True) -> str:
    """libpa.so and, unless `binding` is false, the extension in front of it."""
    if not force and up_to_date():
        if binding:
            build_binding()
        return LIB
    cmd = [_nvcc(), *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-o", LIB, *SOURCES]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    if binding:
        build_binding(force)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv, binding="--library" not in sys.argv)
    print(LIB)
