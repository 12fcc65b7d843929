"""Build the CUDA library ``libmoe.so`` (sm_103a) from ``csrc/`` with nvcc, and
the native part of the Python binding, ``_moe_bind.so``, with the host compiler
against the installed PyTorch.

Each translation unit is compiled in parallel, then linked into one shared
library under ``router_experts_gb300/_build/``.  ``python -m
router_experts_gb300.build`` runs it from the command line.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libmoe.so")
BIND_SRC = os.path.join(CSRC, "bind.cpp")
BIND = os.path.join(BUILD, "_moe_bind.so")
SOURCES = ["api.cu", "router.cu", "align.cu", "ffn.cu", "lowbit.cu", "finalize.cu",
           "router_noalloc.cu", "probe.cu", "decode.cu", "norm.cu", "linear.cu", "balance.cu"]
HEADERS = ["moe_common.cuh", "moe_internal.h", "router_device.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _newer(target: str, files: list) -> bool:
    return os.path.exists(target) and os.path.getmtime(target) >= max(
        os.path.getmtime(f) for f in files)


def _run(cmd: list, what: str, verbose: bool = False):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout, r.stderr, file=sys.stderr)


def _torch_paths():
    """Include directories, library directory and C++ ABI flag of the installed
    PyTorch."""
    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    inc = os.path.join(root, "include")
    return ([inc, os.path.join(inc, "torch", "csrc", "api", "include")], os.path.join(root, "lib"),
            int(torch._C._GLIBCXX_USE_CXX11_ABI))


def _compile_bind(verbose: bool) -> str:
    incs, _, abi = _torch_paths()
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    incs = incs + [cuda, sysconfig.get_paths()["include"]]
    obj = os.path.join(BUILD, "bind.o")
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={abi}", *(f for i in incs for f in ("-isystem", i)),
          "-c", BIND_SRC, "-o", obj], "compiling bind.cpp failed", verbose)
    return obj


def _link_bind(obj: str):
    _, lib, _ = _torch_paths()
    tmp = BIND + f".{os.getpid()}.tmp"
    _run([os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L" + BUILD, "-l:libmoe.so",
          "-L" + lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
          "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib], "linking _moe_bind.so failed")
    os.replace(tmp, BIND)


def build(force: bool = False, verbose: bool = False, extra: list | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    header = os.path.join(HERE, "..", "include", "moe.h")
    inputs = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [header]
    new_lib = force or not _newer(LIB, inputs)
    new_bind = force or not _newer(BIND, [BIND_SRC, header])
    if not new_lib and not new_bind:
        return LIB
    cc = nvcc()
    inc = ["-I", os.path.join(HERE, "..", "include")]

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        _run([cc, *ARCH, *FLAGS, *(extra or []), *inc, "-c", os.path.join(CSRC, src), "-o", obj],
             f"nvcc failed for {src}", verbose)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        bind = ex.submit(_compile_bind, verbose) if new_bind else None
        objs = list(ex.map(compile_one, SOURCES)) if new_lib else []
        bind_obj = bind.result() if bind else None
    if new_lib:
        tmp = LIB + f".{os.getpid()}.tmp"
        _run([cc, *ARCH, "-shared", "-Xlinker", "-soname=libmoe.so", "-o", tmp, *objs],
             "link failed")
        os.replace(tmp, LIB)
    if new_bind:
        _link_bind(bind_obj)
    return LIB


if __name__ == "__main__":
    v = "-v" in sys.argv
    ex = ["-Xptxas", "-v"] if "--ptxas" in sys.argv else None
    print(build(force=True, verbose=v or bool(ex), extra=ex))
