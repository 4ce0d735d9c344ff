"""Build the sm_100a CUDA library ``libmambascan.so`` in-tree with nvcc, and the
Python calls' tensor checks ``_binding.so`` with the host compiler.

Usage: ``python -m selective_state_space_27_b200.build`` (or ``build()``).
The library links the CUDA runtime statically, so it only needs the driver.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libmambascan.so")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_FOR = os.path.join(PKG, "_build", "binding_built_for")   # the torch and Python it was compiled against
SOURCES = ["api.cu", "scan_fwd.cu", "scan_rec.cu", "scan_bwd.cu", "state_update.cu", "noalloc.cu", "ssd_fwd.cu", "probe.cu",
           "conv_packed.cu", "ssd_update.cu", "norm.cu", "ssd_packed.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != "binding.cpp"]
    files.append(os.path.join(INCLUDE, "mambascan.h"))
    files.append(os.path.abspath(__file__))
    return files


def up_to_date() -> bool:
    return _newer(LIB, _inputs())


def _interpreter() -> str:
    """The torch and Python that the binding's machine code has to fit."""
    import torch

    return f"torch {torch.__version__}, Python {sys.version}"


def binding_up_to_date() -> bool:
    try:
        with open(BINDING_FOR) as f:
            if f.read() != _interpreter():
                return False
    except FileNotFoundError:
        return False
    return _newer(BINDING, [os.path.join(CSRC, "binding.cpp"), os.path.join(INCLUDE, "mambascan.h"),
                            os.path.abspath(__file__)])


def _newer(target, files) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(f) <= os.path.getmtime(target) for f in files)


def build_binding(verbose: bool = False) -> str:
    """Compile csrc/binding.cpp against torch's and Python's headers."""
    import torch

    root = os.path.dirname(os.path.abspath(torch.__file__))
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"]]
    tmp = BINDING + f".{os.getpid()}.tmp"
    cmd = [os.environ.get("CXX") or "g++", "-shared", "-fPIC", "-O2", "-std=c++17",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{d}" for d in [INCLUDE, *include]),
           os.path.join(CSRC, "binding.cpp"), "-o", tmp, "-L" + os.path.join(root, "lib"), "-ltorch_python",
           "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, BINDING)
    os.makedirs(os.path.dirname(BINDING_FOR), exist_ok=True)
    with open(BINDING_FOR, "w") as f:
        f.write(_interpreter())
    return BINDING


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile every CUDA source for sm_100a into the in-tree shared library, and, where
    torch is installed, the binding. Returns the library's path."""
    if force or not up_to_date():
        build_library(verbose, ptxas_info)
    try:
        import torch   # noqa: F401
    except ModuleNotFoundError as e:
        if e.name != "torch":
            raise
        print("torch is not installed: only the CUDA library was built, not the Python calls' tensor checks", flush=True)
        return LIB
    if force or not binding_up_to_date():
        build_binding(verbose)
    return LIB


def build_library(verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile every CUDA source for sm_100a into the in-tree shared library."""
    objdir = os.path.join(PKG, "_build")
    os.makedirs(objdir, exist_ok=True)
    common = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]
    if ptxas_info:
        common += ["-Xptxas", "-v"]

    def compile_one(src: str) -> str:
        obj = os.path.join(objdir, src.replace(".cu", ".o"))
        cmd = common + ["-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)
        return obj

    with ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 1)) as pool:
        objs = list(pool.map(compile_one, SOURCES))
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(LIB)
