"""Build the CUDA library libgdr.so in-tree, for sm_103a.

Compiles every ``csrc/*.cu`` with nvcc (``-gencode arch=compute_103a,code=sm_103a``)
in parallel and links them into ``_lib/libgdr.so``. No cmake, no torch
extension machinery: the library has a plain C ABI (``include/gdr.h``).

``csrc/layers_host.cpp``, host code that takes torch tensors to that C ABI, is compiled
beside them with g++ against the installed torch's headers into ``_lib/_layers_host.so``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import importlib.util
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_lib")
OBJ_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libgdr.so")
HOST_SRC = os.path.join(CSRC, "layers_host.cpp")
HOST = os.path.join(OUT_DIR, "_layers_host.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I" + INCLUDE, "-I" + CSRC]


def _nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + [HOST_SRC] + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(INCLUDE, "gdr.h")]


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(HOST):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(HOST))
    return all(os.path.getmtime(d) <= t for d in _deps())


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    return r


def _torch_dir() -> str:
    return os.path.dirname(importlib.util.find_spec("torch").origin)


def _compile_host() -> str:
    torch = os.path.join(_torch_dir(), "include")
    obj = os.path.join(OBJ_DIR, "layers_host.cpp.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-I" + INCLUDE, "-isystem", torch, "-isystem",
          os.path.join(torch, "torch", "csrc", "api", "include"), "-isystem", cuda,
          "-I" + sysconfig.get_paths()["include"], "-c", HOST_SRC, "-o", obj], "g++ on " + HOST_SRC)
    return obj


def _link_host(obj: str) -> None:
    libs = os.path.join(_torch_dir(), "lib")
    tmp = HOST + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, "-L" + libs, "-ltorch_python", "-ltorch", "-ltorch_cpu",
          "-ltorch_cuda", "-lc10", "-lc10_cuda", "-L" + OUT_DIR, "-lgdr", "-Wl,-rpath," + libs,
          "-Wl,-rpath,$ORIGIN"], "link of " + HOST)
    os.replace(tmp, HOST)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(OUT_DIR, exist_ok=True)
    os.makedirs(OBJ_DIR, exist_ok=True)
    srcs = _sources()

    def compile_one(src):
        obj = os.path.join(OBJ_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(16, len(srcs) + 1)) as ex:
        host = ex.submit(_compile_host)
        objs = list(ex.map(compile_one, srcs))
        host_obj = host.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs, "-ldl", "-lrt", "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_host(host_obj)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
