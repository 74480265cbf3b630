"""Builds ``libgbr.so`` (the C-ABI library of this package) with nvcc, and the
compiled Python binding of the feed-forward operators with the host compiler.

Every translation unit under ``csrc/`` is compiled for sm_103a only, in
parallel, then linked into one shared library next to this file.
``csrc/python/operators_ext.cpp`` becomes ``_operators_ext.so``, the only part
that is compiled against PyTorch; it is linked to ``libgbr.so``.  The results
are git-ignored and rebuilt on each machine (they are specific to the host's
architecture and to its PyTorch).

The library needs nvcc alone and is linked first.  Where PyTorch, its headers
or Python's are missing, the binding is left out, with a warning.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sysconfig
import warnings

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ_DIR = os.path.join(PKG_DIR, "_build")
LIB_PATH = os.path.join(PKG_DIR, "libgbr.so")
EXT_SRC = os.path.join(CSRC, "python", "operators_ext.cpp")
EXT_PATH = os.path.join(PKG_DIR, "_operators_ext.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-I" + CSRC, "-I" + INCLUDE]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA 13 toolkit is required to build libgbr.so")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [EXT_SRC, os.path.abspath(__file__)])


def _torch_dir():
    spec = importlib.util.find_spec("torch")
    return list(spec.submodule_search_locations)[0] if spec is not None and spec.submodule_search_locations else None


def binding_lacks():
    """What the Python binding cannot be compiled without and is not there, or None."""
    torch_dir = _torch_dir()
    if torch_dir is None:
        return "PyTorch"
    if not os.path.exists(os.path.join(torch_dir, "include", "ATen", "ATen.h")):
        return "PyTorch's headers"
    if not os.path.exists(os.path.join(torch_dir, "lib", "libc10_cuda.so")):
        return "PyTorch for CUDA"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python.h"
    return None


def up_to_date() -> bool:
    made = [LIB_PATH] if binding_lacks() else [LIB_PATH, EXT_PATH]
    if not all(os.path.exists(p) for p in made):
        return False
    t = min(os.path.getmtime(p) for p in made)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _compile_ext(obj: str, torch_dir: str) -> None:
    """Compiles the Python binding to an object file."""
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    include = [INCLUDE, os.path.join(torch_dir, "include"),
               os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    cmd = (["g++", "-O2", "-std=c++17", "-fPIC", "-c", EXT_SRC, "-o", obj] + ["-I" + i for i in include])
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed for %s:\n%s\n%s" % (EXT_SRC, res.stdout, res.stderr))


def _link_ext(obj: str, torch_dir: str) -> None:
    tmp = EXT_PATH + ".tmp%d" % os.getpid()
    lib = os.path.join(torch_dir, "lib")
    cmd = ["g++", "-shared", "-o", tmp, obj, LIB_PATH, "-Wl,-rpath,$ORIGIN", "-L" + lib, "-ltorch_python", "-ltorch",
           "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link of the Python binding failed:\n%s\n%s" % (res.stdout, res.stderr))
    os.replace(tmp, EXT_PATH)


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile and link; returns the library path."""
    if not force and up_to_date():
        return LIB_PATH
    lacks, torch_dir = binding_lacks(), _torch_dir()
    if lacks:
        warnings.warn("the Python binding of the feed-forward operators is not built: %s not found" % lacks)
    nvcc = _nvcc()
    os.makedirs(OBJ_DIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []

    def compile_one(src):
        obj = os.path.join(OBJ_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc] + NVCC_FLAGS + extra + ["-c", src, "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, res.stdout, res.stderr))
        return obj, res.stderr

    srcs = _sources()
    ext_obj = os.path.join(OBJ_DIR, "operators_ext.o")
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        ext = None if lacks else ex.submit(_compile_ext, ext_obj, torch_dir)
        results = list(ex.map(compile_one, srcs))
    if verbose or ptxas_verbose:
        for _, log in results:
            if log.strip():
                print(log)
    tmp = LIB_PATH + ".tmp%d" % os.getpid()
    cmd = [nvcc] + ARCH + ["-shared", "-Xlinker", "-soname=libgbr.so", "-o", tmp] + [o for o, _ in results]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (res.stdout, res.stderr))
    os.replace(tmp, LIB_PATH)
    if ext is not None:
        ext.result()
        _link_ext(ext_obj, torch_dir)
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv))
