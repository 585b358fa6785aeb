"""Build libmoe_routing.so (sm_100a) in-tree with nvcc, and the native part of
the Python binding (_experts.so).

Usage: ``python -m moe_expert_routing_token_b200.build`` (or call
:func:`build`).  Both land in ``moe_expert_routing_token_b200/_lib/`` next to
the binding that loads them.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_DIR = os.path.join(PKG, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libmoe_routing.so")
BINDING = os.path.join(CSRC, "binding.cpp")
BINDING_PATH = os.path.join(LIB_DIR, "_experts.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-std=c++17", "-lineinfo",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return _older(LIB_PATH, deps)


def _older(path: str, deps: list[str]) -> bool:
    return not os.path.exists(path) or any(os.path.getmtime(d) > os.path.getmtime(path) for d in deps)


def _binding_stale() -> bool:
    return _older(BINDING_PATH, [BINDING] + glob.glob(os.path.join(INCLUDE, "*.h")))


def _binding_command(out: str) -> list[str]:
    # nvcc as the driver: the host compiler, and with it the C++ runtime that
    # torch's exceptions cross, is then the library's own
    home = os.path.dirname(torch.__file__)
    return [os.environ.get("NVCC", "nvcc"), "-O2", "-std=c++17", "-shared", "-cudart", "none",
            "-gencode", "arch=compute_100a,code=sm_100a", "-Xcompiler", "-fPIC,-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
            "-I", os.path.join(home, "include"),
            "-I", os.path.join(home, "include", "torch", "csrc", "api", "include"),
            "-I", sysconfig.get_paths()["include"], BINDING, "-o", out,
            "-L", os.path.join(home, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
            LIB_PATH, "-Xlinker", "-rpath,$ORIGIN"]


def build(force: bool = False, verbose: bool = False, jobs: int = 8) -> str:
    """Compile every CUDA source for sm_100a, link the shared library, and
    compile the binding against it."""
    if force or _stale():
        _build_library(verbose, jobs)
    if force or _binding_stale():
        tmp = BINDING_PATH + f".tmp{os.getpid()}"
        subprocess.run(_binding_command(tmp), check=True)
        os.replace(tmp, BINDING_PATH)
    return LIB_PATH


def _build_library(verbose: bool, jobs: int) -> None:
    nvcc = os.environ.get("NVCC", "nvcc")
    obj_dir = os.path.join(PKG, "_build")
    os.makedirs(obj_dir, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    procs = []
    objs = []
    for src in sources():
        obj = os.path.join(obj_dir, os.path.basename(src) + ".o")
        objs.append(obj)
        cmd = [nvcc, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                                            text=True)))
        if len(procs) >= jobs:
            _drain(procs, verbose)
    _drain(procs, verbose)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    subprocess.run([nvcc, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", *objs,
                    "-Xlinker", "-soname=libmoe_routing.so", "-o", tmp], check=True)
    os.replace(tmp, LIB_PATH)


def _drain(procs, verbose):
    while procs:
        cmd, p = procs.pop(0)
        out, _ = p.communicate()
        if verbose or p.returncode != 0:
            sys.stdout.write(out)
        if p.returncode != 0:
            raise RuntimeError("nvcc failed: " + " ".join(cmd))


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
