"""Builds libmxnorm_b200.so in-tree with nvcc for sm_100a (no JIT cache), and where
torch is installed the Python module that marshals its tensors (host code only).

    python -m normalisation_row_bf16_b200.build
"""
from __future__ import annotations

import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libmxnorm_b200.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC", "-Xptxas", "-warn-spills"]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def _older(target: str, srcs) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(s) > t for s in srcs)


def is_stale() -> bool:
    return _older(LIB, sources())


def has_torch() -> bool:
    return importlib.util.find_spec("torch") is not None


def binding_path() -> str:
    """The binding module for this interpreter and this torch: it is compiled
    against the headers of both, so another version's is not loaded."""
    import torch

    return os.path.join(PKG, f"_binding.torch-{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")


def binding_is_stale() -> bool:
    return _older(binding_path(), [BINDING_SRC] + glob.glob(os.path.join(INCLUDE, "*.h")))


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _start_binding(verbose: bool):
    """Starts the compiler on the binding module: (process, temporary output)."""
    import torch
    from torch.utils import cpp_extension

    tmp = binding_path() + f".tmp{os.getpid()}"
    inc = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    inc += cpp_extension.include_paths()
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *["-I" + i for i in inc], "-o", tmp, BINDING_SRC,
           "-L" + lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    return subprocess.Popen(cmd), tmp


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every translation unit in csrc/ (in parallel) and link the
    library, and the binding module beside it.  The library does not depend on
    torch: without it, or where the binding does not compile, it is built all the
    same (and the failure raised after it)."""
    binding = why = None
    if not has_torch():
        if verbose:
            print("no torch: building the library without its Python binding", file=sys.stderr)
    else:
        try:
            if force or binding_is_stale():
                binding = _start_binding(verbose)
        except Exception as e:  # noqa: BLE001 -- a broken torch or no C++ compiler
            why = e
    try:
        lib = _build_library(force, verbose)
    finally:
        if binding:
            if binding[0].wait() == 0:
                os.replace(binding[1], binding_path())
            else:
                why = RuntimeError("the compiler failed")
    if why is not None:
        raise RuntimeError("the binding module was not built") from why
    return lib


def _build_library(force: bool, verbose: bool) -> str:
    if not force and not is_stale():
        return LIB
    tus = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    objdir = os.path.join(PKG, "_build")
    os.makedirs(objdir, exist_ok=True)
    procs = []
    for tu in tus:
        obj = os.path.join(objdir, os.path.basename(tu) + f".{os.getpid()}.o")
        cmd = [nvcc(), *NVCC_FLAGS, "-c", "-I" + INCLUDE, "-o", obj, tu]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((obj, subprocess.Popen(cmd)))
    objs = []
    failed = False
    for obj, p in procs:
        failed |= p.wait() != 0
        objs.append(obj)
    if failed:
        raise RuntimeError("nvcc failed")
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run([nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp, *objs], check=True)
    os.replace(tmp, LIB)
    for o in objs:
        os.remove(o)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
