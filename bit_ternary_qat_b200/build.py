"""Build libbitlinear.so in-tree with nvcc for sm_100a (no JIT cache, no torch extension).

    python -m bit_ternary_qat_b200.build [--force]
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC_DIR = os.path.join(HERE, "csrc")
MAIN = os.path.join(SRC_DIR, "bitlinear.cu")
HEADER = os.path.join(ROOT, "include", "bitlinear.h")
LIB = os.path.join(HERE, "libbitlinear.so")
MARSHAL_SRC = os.path.join(SRC_DIR, "marshal.cpp")
MARSHAL = os.path.join(HERE, "_marshal.so")      # tensor-level calls in C++, over libbitlinear.so's C ABI

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "-Xcompiler", "-fvisibility=hidden",
]


def _sources():
    out = [HEADER]
    for f in sorted(os.listdir(SRC_DIR)):
        if f.endswith((".cu", ".cuh")):
            out.append(os.path.join(SRC_DIR, f))
    return out


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(s) <= t for s in _sources())


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def _torch_mark() -> bytes:
    """What a _marshal.so built against the installed torch and Python holds (torch's C++ classes
    change from release to release)."""
    import torch
    return ("bitlinear binding for torch %s, Python %d.%d;" % (torch.__version__, *sys.version_info[:2])).encode()


def marshal_fits() -> bool:
    """Whether _marshal.so was built against the installed torch."""
    with open(MARSHAL, "rb") as f:
        return _torch_mark() in f.read()


def build_marshal(force: bool = False, verbose: bool = False) -> str:
    """The C++ part of the binding (g++, against the installed torch)."""
    if not force and os.path.exists(MARSHAL) and all(
            os.path.getmtime(s) <= os.path.getmtime(MARSHAL) for s in (MARSHAL_SRC, HEADER)) and marshal_fits():
        return MARSHAL
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = MARSHAL + ".tmp.%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
           '-DBL_TORCH_MARK="%s"' % _torch_mark().decode(),
           *[a for d in cpp_extension.include_paths() for a in ("-isystem", d)],
           "-isystem", os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"),
           "-isystem", sysconfig.get_paths()["include"], MARSHAL_SRC, "-o", tmp,
           "-L", lib, "-Wl,-rpath," + lib, "-lc10", "-lc10_cuda", "-ltorch_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, MARSHAL)
    return MARSHAL


def build_lib(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [nvcc(), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), MAIN, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


def build(force: bool = False, verbose: bool = False) -> str:
    """The library, then the binding's C++ part: where that cannot be built (no torch headers) this
    raises, with the library in place for the calls that need nothing else."""
    build_lib(force, verbose)
    build_marshal(force, verbose)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
