"""Build ``libmoe.so`` (the C-ABI library) in-tree for sm_100a with nvcc, and
``_torch_binding.so`` (the compiled Python calls of its 8-bit entry points)
with g++ against the installed torch.

Run as ``python -m moe_routing_expert_fp32_b200.build [--force] [-v]``.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libmoe.so")
BINDING = os.path.join(HERE, "_torch_binding.so")
BINDING_SRC = os.path.join(CSRC, "torch_binding.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17", "-shared",
    "-Xcompiler", "-fPIC,-fvisibility=hidden",
    "-I", INCLUDE, "-I", CSRC,
]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(INCLUDE, "moe.h")]
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and not _stale():
        build_binding(verbose=verbose)
        return LIB
    cmd = ["nvcc", *NVCC_FLAGS]
    if ptxas_info:
        cmd += ["-Xptxas", "-v"]
    cmd += [*sources(), "-o", LIB]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    build_binding(force=force, verbose=verbose)
    return LIB


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """The compiled Python calls; libmoe.so must exist (they link to it)."""
    deps = (BINDING_SRC, os.path.join(INCLUDE, "moe.h"))
    if not force and os.path.exists(BINDING) and all(
            os.path.getmtime(p) <= os.path.getmtime(BINDING) for p in deps):
        return BINDING
    import torch
    t = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-isystem", os.path.join(t, "include"),
           "-isystem", os.path.join(t, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(cuda, "include"), BINDING_SRC, "-o", BINDING,
           "-L", HERE, "-l:libmoe.so", "-Wl,-rpath,$ORIGIN", "-L", os.path.join(t, "lib"),
           "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    return BINDING


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                ptxas_info="--ptxas" in sys.argv))
