"""Builds libgspn.so in-tree with nvcc for sm_100a (B200). No torch types cross the C ABI."""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libgspn.so")
BINDING_SRC = os.path.join(CSRC, "seq_binding.cpp")
BINDING = os.path.join(HERE, "_seq_fast.so")

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def _older(target: str, sources) -> bool:
    return not os.path.exists(target) or any(os.path.getmtime(f) > os.path.getmtime(target) for f in sources)


def stale() -> bool:
    return _older(LIB, sources() + headers() + [__file__])


def binding_stale() -> bool:
    return _older(BINDING, headers() + [BINDING_SRC, __file__])


def binding_command(out: str):
    """g++ for the binding of the token-sequence calls: a CPython module against torch's headers, which
    calls libgspn's entry points by address."""
    import sysconfig

    import torch

    troot = os.path.dirname(torch.__file__)
    inc = [os.path.join(troot, "include"), os.path.join(troot, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include"), sysconfig.get_paths()["include"]]
    lib = os.path.join(troot, "lib")
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f for p in inc for f in ("-isystem", p)],
            "-I", INCLUDE, BINDING_SRC, "-o", out, "-L", lib, "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]


def _start_binding(out: str):
    try:
        return subprocess.Popen(binding_command(out))
    except OSError:                      # no such compiler
        return None


def _finish_binding(process, out: str):
    """Without the binding every call goes through the checks in Python: the same results, some 20 us a call later.
    An older one is taken away, since it may disagree with the library about what they pass each other."""
    if process is not None and process.wait() == 0:
        os.replace(out, BINDING)
        return
    for f in (out, BINDING):
        if os.path.exists(f):
            os.remove(f)
    warnings.warn(f"{os.path.basename(BINDING)} was not built (a C++ compiler, Python's and torch's headers are needed): "
                  "token-sequence calls take the slower path through Python", RuntimeWarning, stacklevel=3)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Compiles libgspn.so, and the native binding of the token-sequence calls where that is possible."""
    binding = None
    if force or binding_stale():
        tmp_binding = BINDING + f".tmp{os.getpid()}"
        binding = (_start_binding(tmp_binding), tmp_binding)
    if force or stale():
        try:
            _build_library(verbose, extra)
        except BaseException:
            if binding and binding[0]:
                binding[0].kill()
                binding[0].wait()
                if os.path.exists(binding[1]):
                    os.remove(binding[1])
            raise
    if binding:
        _finish_binding(*binding)
    return LIB


def _build_library(verbose, extra):
    nvcc = os.environ.get("NVCC", "nvcc")
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    procs = []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [nvcc, *NVCC_FLAGS, *extra, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((subprocess.Popen(cmd), src))
        objs.append(obj)
    for p, src in procs:
        if p.wait() != 0:
            raise RuntimeError(f"nvcc failed on {src}")
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([nvcc, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", "-o", tmp, *objs])
    os.replace(tmp, LIB)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)
