"""Build libgbattn.so in-tree with nvcc for sm_103a, and the Python extension
that calls it.

Each translation unit under csrc/ is compiled in parallel to an object in
``_build/`` and linked (static CUDA runtime) into ``lib/libgbattn.so``.  A
unit is recompiled only when it or a header is newer than its object.
``csrc/binding.cpp`` (host code against PyTorch's headers) becomes
``lib/_binding.so`` beside it.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import platform
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
MACHINE = platform.machine()
BUILD = os.path.join(PKG, "_build", MACHINE)   # objects differ per host architecture
LIB_DIR = os.path.join(PKG, "lib")
LIB_PATH = os.path.join(LIB_DIR, "libgbattn.so")
STAMP = LIB_PATH + ".machine"
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING_PATH = os.path.join(LIB_DIR, "_binding.so")
BINDING_STAMP = BINDING_PATH + ".machine"

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libgbattn")
    return path


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    newest = max([os.path.getmtime(src)] + [os.path.getmtime(h) for h in _headers()])
    if os.path.exists(obj) and os.path.getmtime(obj) >= newest:
        return obj
    cmd = [nvcc()] + ARCH + NVCC_FLAGS + ["-c", src, "-o", obj + ".tmp"]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{res.stdout}\n{res.stderr}")
    if verbose_ptxas and res.stderr:
        print(res.stderr)
    os.replace(obj + ".tmp", obj)
    return obj


def _build_binding() -> None:
    """lib/_binding.so for this machine, Python and PyTorch."""
    import torch
    made_for = " ".join((MACHINE, platform.python_version(), torch.__version__))
    header = os.path.join(INCLUDE, "gbattn.h")
    if (os.path.exists(BINDING_PATH) and os.path.exists(BINDING_STAMP)
            and open(BINDING_STAMP).read().strip() == made_for
            and os.path.getmtime(BINDING_PATH) >= max(os.path.getmtime(BINDING_SRC),
                                                      os.path.getmtime(header))):
        return
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           "-I", os.path.join(root, "include"),
           "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"), BINDING_SRC,
           "-o", tmp, "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu",
           "-lc10", "-lc10_cuda"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        for stale in (BINDING_STAMP, BINDING_PATH):   # of an older header, perhaps
            if os.path.exists(stale):
                os.remove(stale)
        raise RuntimeError(f"g++ failed on binding.cpp:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, BINDING_PATH)
    with open(BINDING_STAMP, "w") as f:
        f.write(made_for)


def build(verbose_ptxas: bool = False) -> str:
    """Compile every .cu under csrc/, link lib/libgbattn.so and build the
    extension; returns the library's path.  An extension that does not compile
    raises too, but only once the library stands: all but the paged-cache
    functions work without it."""
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs)) + 1) as ex:
        binding = ex.submit(_build_binding)
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs))
    newest = max(os.path.getmtime(o) for o in objs)
    stamp_ok = os.path.exists(STAMP) and open(STAMP).read().strip() == MACHINE
    if not (stamp_ok and os.path.exists(LIB_PATH) and os.path.getmtime(LIB_PATH) >= newest):
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        cmd = [nvcc()] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
        os.replace(tmp, LIB_PATH)
        with open(STAMP, "w") as f:
            f.write(MACHINE)
    binding.result()
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(verbose_ptxas="-v" in sys.argv))
