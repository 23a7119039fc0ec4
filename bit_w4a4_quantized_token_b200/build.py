"""Compile the CUDA library (sm_100a) in-tree, libsvdq_b200.so next to this file,
and the CPython module beside it that makes the W8A8 layer's calls (_w8a8_front.<torch and
Python it was built for>.so).

    python -m bit_w4a4_quantized_token_b200.build [--force]
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys

_HERE = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_HERE)
LIB = os.path.join(_HERE, "libsvdq_b200.so")
SOURCES = sorted(glob.glob(os.path.join(_HERE, "csrc", "*.cu")) + glob.glob(os.path.join(_HERE, "csrc", "*.cuh"))
                 + glob.glob(os.path.join(_HERE, "csrc", "*.h")) + [os.path.join(_ROOT, "include", "svdq.h")])
MAIN = os.path.join(_HERE, "csrc", "svdq_lib.cu")
FRONT_MAIN = os.path.join(_HERE, "csrc", "w8a8_front.cpp")


def nvcc_command(out: str = LIB) -> list[str]:
    nvcc = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
    return [nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
            "-Xcompiler", "-fPIC", "-shared", "-I" + os.path.join(_ROOT, "include"), "-o", out, MAIN]


def front_path() -> str:
    """The native module's file for the running Python and torch: its name holds both, because it is compiled against
    the C++ of the one and the C API of the other and is of no use to any other pair."""
    import sysconfig

    import torch

    return os.path.join(_HERE, f"_w8a8_front.torch-{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")


def front_command(out: str) -> list[str]:
    import sysconfig

    import torch

    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-I" + os.path.join(_ROOT, "include"), "-I" + sysconfig.get_paths()["include"], "-isystem", inc, "-isystem",
            os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", "/usr/local/cuda/include", "-o", out,
            FRONT_MAIN, "-L" + lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-ltorch",
            # the C++ runtime that torch has loaded, also where the compiler would link its own statically: streams
            # and exceptions pass between the two
            "-l:libstdc++.so.6"]


def _compile(out: str, sources: list[str], command, force: bool, verbose: bool) -> str:
    if not force and os.path.exists(out) and os.path.getmtime(out) >= max(os.path.getmtime(s) for s in sources):
        return out
    tmp = out + f".tmp{os.getpid()}"
    cmd = command(tmp)
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, out)
    return out


def front_lacks() -> str:
    """What the native module needs and this machine does not have ("" when it has all)."""
    import importlib.util
    import sysconfig

    spec = importlib.util.find_spec("torch")
    if spec is None:
        return "torch"
    if not os.path.exists(os.path.join(spec.submodule_search_locations[0], "lib", "libc10_cuda.so")):
        return "a torch with CUDA"
    return "" if os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")) else "Python's headers"


def build(force: bool = False, verbose: bool = False) -> str:
    """The library first: it needs no more than nvcc, and neither do the C ABI's users."""
    lib = _compile(LIB, SOURCES, nvcc_command, force, verbose)
    lacking = front_lacks()
    if lacking:
        print(f"the W8A8 layer's Python module is not built: no {lacking}", file=sys.stderr)
    else:
        _compile(front_path(), [FRONT_MAIN, os.path.join(_ROOT, "include", "svdq.h")], front_command, force, verbose)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
