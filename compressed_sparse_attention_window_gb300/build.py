"""Build ``libds41.so`` (the CUDA path) in-tree with nvcc for sm_103a.

Each ``csrc/*.cu`` compiles to an object in parallel, then nvcc links the
shared library next to this file.  No fast-math: the fp4 quantisers and the
indexer scores must round exactly as IEEE single precision does.  The host
compiler builds ``csrc/ds41_binding.cpp``, the extension module with the
Python side of the dense attention's calls, against the installed torch.

Usage: ``python -m compressed_sparse_attention_window_gb300.build [--force]``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libds41.so")
BINDING_SRC = os.path.join(CSRC, "ds41_binding.cpp")
BINDING = os.path.join(HERE, "_ds41_binding.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
                     "-I", CSRC, "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libds41")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    if _stale(obj, [src] + _headers() + [__file__]):
        cmd = [nvcc(), *NVCC_FLAGS, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
    return obj


def _build_binding(force: bool, verbose: bool) -> None:
    """The extension module (its libraries are those that torch has loaded).  It is
    stale, too, when the torch, the Python or the command it was built with change."""
    import torch
    cxx = shutil.which("g++") or "g++"
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    dirs = [INCLUDE, os.path.join(root, "include"), sysconfig.get_paths()["include"],
            os.path.join(cuda, "include")]
    tmp = BINDING + f".{os.getpid()}.tmp"
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *(x for d in dirs for x in ("-I", d)), BINDING_SRC,
           "-L", os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch",
           "-ltorch_python"]
    made_with = "\n".join([torch.__version__, sysconfig.get_config_var("SOABI") or "", *cmd])
    stamp = os.path.join(BUILD, "binding.txt")
    if not (force or _stale(BINDING, [BINDING_SRC, __file__] + _headers())):
        if os.path.exists(stamp) and open(stamp).read() == made_with:
            return
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd + ["-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cxx} failed for {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(stamp, "w") as f:
        f.write(made_with)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every CUDA source, link libds41.so and build the extension module;
    returns the library's path."""
    os.makedirs(BUILD, exist_ok=True)
    if force:
        for o in glob.glob(os.path.join(BUILD, "*.o")):
            os.remove(o)
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs)) + 1) as ex:
        binding = ex.submit(_build_binding, force, verbose)
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
        binding.result()
    if force or _stale(LIB, objs):
        tmp = LIB + f".{os.getpid()}.tmp"
        cuda_lib = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "lib64")
        cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-lcudart",
               "-Xlinker", "-rpath", "-Xlinker", cuda_lib]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
