"""Build the CUDA library in-tree: bit_mla_kv_qdecode_b200/lib/libmla_qcache.so.

nvcc compiles every csrc/*.cu for sm_100a only (B200), links them into one
shared library with a C ABI (include/mla_qcache.h), and needs no GPU. Where
PyTorch is installed, its binding of the operators around the decode
(csrc/torch_binding.cpp) is built beside it and linked against it.

    python -m bit_mla_kv_qdecode_b200.build [--verbose]
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB_DIR = os.path.join(PKG, "lib")
LIB_PATH = os.path.join(LIB_DIR, "libmla_qcache.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def binding_path() -> str:
    """Where the binding for the installed PyTorch is: its name carries the versions whose binary interface it is
    compiled for, so that another PyTorch's or Python's is not taken for it."""
    import torch
    return os.path.join(LIB_DIR, f"_mla_torch-{torch.__version__}-{sys.implementation.cache_tag}.so")


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def sources():
    return sorted(glob.glob(os.path.join(PKG, "csrc", "*.cu")))


def build(verbose: bool = False, force: bool = False) -> str:
    srcs = sources()
    deps = srcs + glob.glob(os.path.join(PKG, "csrc", "*.h")) + glob.glob(os.path.join(PKG, "csrc", "*.cuh")) \
        + glob.glob(os.path.join(ROOT, "include", "*.h"))
    if not force and os.path.exists(LIB_PATH):
        newest = max(os.path.getmtime(p) for p in deps)
        if os.path.getmtime(LIB_PATH) >= newest:
            build_binding(verbose)
            return LIB_PATH
    os.makedirs(LIB_DIR, exist_ok=True)
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc_path(), *ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-shared",
           "-I", os.path.join(ROOT, "include"), "-Xptxas", "-v" if verbose else "-O3",
           *srcs, "-o", tmp]
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + proc.stdout + proc.stderr)
    if verbose:
        sys.stdout.write(proc.stdout + proc.stderr)
    os.replace(tmp, LIB_PATH)
    build_binding(verbose, force)
    return LIB_PATH


def build_binding(verbose: bool = False, force: bool = False) -> None:
    """The binding, where PyTorch is installed. The library stands without it: where it cannot be built (no C++
    compiler, no CUDA headers, a PyTorch without CUDA), that is a warning here and an ImportError at its first use."""
    try:
        import torch
    except ImportError:
        return  # the C ABI and its ctypes binding stand alone
    src, header = os.path.join(PKG, "csrc", "torch_binding.cpp"), os.path.join(ROOT, "include", "mla_qcache.h")
    path = binding_path()
    if not force and os.path.exists(path) and os.path.getmtime(path) >= max(os.path.getmtime(src), os.path.getmtime(header)):
        return
    where = os.path.dirname(torch.__file__)
    tmp = path + ".tmp"
    try:
        cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
        cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
               "-I", os.path.join(ROOT, "include"), "-I", os.path.join(where, "include"),
               "-I", os.path.join(where, "include", "torch", "csrc", "api", "include"),
               "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"), src, "-o", tmp,
               "-L", LIB_DIR, "-lmla_qcache", "-Wl,-rpath,$ORIGIN",
               "-L", os.path.join(where, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
        proc = subprocess.run(cmd, capture_output=True, text=True)
        why = proc.stdout + proc.stderr if proc.returncode != 0 else None
    except (OSError, RuntimeError) as e:
        why = str(e)
    if why is not None:
        if os.path.exists(path):
            os.remove(path)  # of older sources
        warnings.warn(f"{LIB_PATH} is built, its PyTorch binding is not; api's operators around the decode need it:\n{why}")
        return
    if verbose:
        sys.stdout.write(proc.stdout + proc.stderr)
    os.replace(tmp, path)


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv, force=True))
