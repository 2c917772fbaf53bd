"""Build libmoe_b200.so in-tree for sm_100a with nvcc, and the native part of its Python binding
(_moe_ops.so, against the installed torch) with g++.

    python -m fp8_fp4_moe_b200.build [--force] [--verbose]

The library is the product: every step of the layer runs in its kernels.  It
links the CUDA runtime statically and reaches the driver only through
cudaGetDriverEntryPoint, so loading it needs no GPU.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libmoe_b200.so")
OPS = os.path.join(PKG, "_moe_ops.so")
OPS_SOURCE = "ops_binding.cpp"
BUILD_DIR = os.path.join(ROOT, "_build")
OPS_STAMP = os.path.join(BUILD_DIR, "_moe_ops.txt")
SOURCES = ["gemm_sm100.cu", "path_kernels.cu", "moe_api.cu", "noalloc.cu", "dense_api.cu", "gemm_fp8.cu", "quant_fp8.cu",
           "balance.cu"]
HEADERS = ["common.cuh", "kernels.h", "path_phases.cuh"]

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-v", "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found")
    return exe


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every CUDA source for sm_100a and link the shared library. Returns its path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(INCLUDE, "moe_b200.h")]
    objs = []
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + hdrs):
            jobs.append([nvcc(), *ARCH, *FLAGS, "-c", s, "-o", o])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        for cmd, r in ex.map(run, jobs):
            if verbose or r.returncode != 0:
                sys.stderr.write(r.stdout + r.stderr)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed: {' '.join(cmd)}")
    if force or _stale(LIB, objs):
        cmd = [nvcc(), *ARCH, "-shared", "-o", LIB, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link failed")
    missing = ops_prerequisites()
    if missing:   # the library is complete without it; the functions that need it say so when they are called
        warnings.warn(f"{os.path.basename(OPS)} not built, missing: {', '.join(missing)}")
    else:
        build_ops(force, verbose)
    return LIB


def ops_prerequisites() -> list:
    """What the native part of the binding needs and this machine lacks."""
    try:
        import torch
    except ImportError:
        return ["torch"]
    need = [os.path.join(sysconfig.get_path("include"), "Python.h"),
            os.path.join(os.path.dirname(torch.__file__), "include", "torch", "csrc", "autograd", "python_variable.h")]
    return [p for p in need if not os.path.exists(p)] + ([] if shutil.which("g++") else ["g++"])


def _built_for() -> str:
    """The interpreter and torch whose C++ interface _moe_ops.so is compiled against."""
    import torch
    return f"Python {sys.version}, torch {torch.__version__} at {os.path.dirname(torch.__file__)}"


def ops_stale() -> bool:
    """Whether _moe_ops.so is missing, older than its sources, or built for another interpreter or torch."""
    if _stale(OPS, [os.path.join(CSRC, OPS_SOURCE), os.path.join(INCLUDE, "moe_b200.h")]):
        return True
    if not os.path.exists(OPS_STAMP):
        return True
    with open(OPS_STAMP) as f:
        return f.read() != _built_for()


def build_ops(force: bool = False, verbose: bool = False) -> str:
    """Compile the native part of the binding; it finds libmoe_b200.so beside itself, torch's libraries in
    the process that imported torch."""
    import torch
    if not force and not ops_stale():
        return OPS
    src = os.path.join(CSRC, OPS_SOURCE)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    at = os.path.dirname(torch.__file__)
    inc = ["-I" + p for p in [INCLUDE, sysconfig.get_path("include"), os.path.join(cuda, "include"),
                              os.path.join(at, "include"), os.path.join(at, "include", "torch", "csrc", "api", "include")]]
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", *inc, src, "-o", OPS,
           "-L" + PKG, "-lmoe_b200", "-Wl,-rpath,$ORIGIN", "-L" + os.path.join(at, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu",
           "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed: {' '.join(cmd)}")
    os.makedirs(BUILD_DIR, exist_ok=True)
    with open(OPS_STAMP, "w") as f:
        f.write(_built_for())
    return OPS


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
