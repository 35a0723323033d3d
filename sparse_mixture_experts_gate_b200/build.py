"""Build libmoe.so (the C ABI of include/moe.h) for sm_100a with nvcc, and _operators.so
(the torch side of operators.py) with the host compiler, in-tree.

    python -m sparse_mixture_experts_gate_b200.build [--force]

Each .cu under csrc/ is compiled to an object file with
`-gencode arch=compute_100a,code=sm_100a -O3 -lineinfo`, in parallel, and linked
into sparse_mixture_experts_gate_b200/libmoe.so with the CUDA runtime linked
statically (the driver library is loaded at run time). csrc/operators_torch.cpp is
compiled against torch's headers and linked with libmoe.so beside it.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG, "libmoe.so")
OPERATORS_SRC = os.path.join(CSRC, "operators_torch.cpp")
OPERATORS_PATH = os.path.join(PKG, "_operators.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(p) <= t for p in _deps())


def build_operators(force: bool = False) -> str:
    """_operators.so, after libmoe.so, which it is linked with."""
    import sysconfig
    import torch
    deps = [OPERATORS_SRC, os.path.join(INCLUDE, "moe.h"), os.path.abspath(__file__)]
    if not force and os.path.exists(OPERATORS_PATH) and \
            all(os.path.getmtime(p) <= os.path.getmtime(OPERATORS_PATH) for p in deps):
        return OPERATORS_PATH
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    headers = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        raise RuntimeError("no host C++ compiler found")
    tmp = OPERATORS_PATH + f".tmp{os.getpid()}"
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-shared", "-DTORCH_EXTENSION_NAME=_operators",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           *[a for h in headers for a in ("-isystem", h)], OPERATORS_SRC, "-o", tmp, "-L" + os.path.join(root, "lib"),
           "-lc10", "-ltorch_cpu", "-ltorch_cuda", "-lc10_cuda", "-ltorch_python", "-L" + PKG, "-l:libmoe.so",
           "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cxx} failed for {OPERATORS_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, OPERATORS_PATH)
    return OPERATORS_PATH


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and up_to_date():
        build_operators()
        return LIB_PATH
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
                    "-I", INCLUDE, "-I", CSRC, *extra_flags]

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [cc, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, _sources()))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    build_operators(force)
    return LIB_PATH


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
    print(LIB_PATH)
