"""Build the CUDA library libgdr.so in-tree, for sm_103a.

Compiles every ``csrc/*.cu`` with nvcc (``-gencode arch=compute_103a,code=sm_103a``)
in parallel and links them into ``_lib/libgdr.so``. No cmake, no torch
extension machinery: the library has a plain C ABI (``include/gdr.h``).

``csrc/layers_host.cpp``, host code that takes torch tensors to that C ABI, is compiled
beside them with g++ against the installed torch's headers. It fits that torch alone, so
its file is named after torch's version (host_path). It is an extra: the library builds
without torch's headers or g++, and ``layers.py`` then makes its calls from Python.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_lib")
OBJ_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libgdr.so")
HOST_SRC = os.path.join(CSRC, "layers_host.cpp")
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


HEADER = os.path.join(INCLUDE, "gdr.h")


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [HEADER]


def _fresh(path, deps) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(d) <= os.path.getmtime(path) for d in deps)


def host_path(version: str) -> str:
    """The compiled calls of layers.py for this torch and this Python."""
    return os.path.join(OUT_DIR, f"_layers_host-{version}-{sysconfig.get_config_var('SOABI')}.so")


def _torch_dir():
    """Where torch is installed, or None."""
    spec = importlib.util.find_spec("torch")
    return spec and os.path.dirname(spec.origin)


def _host_target():
    """host_path of the installed torch (which need not be imported), or None without one."""
    torch = _torch_dir()
    if not torch:
        return None
    with open(os.path.join(torch, "version.py")) as f:
        version = re.search(r"""__version__ = ['"]([^'"]+)""", f.read())
    return version and host_path(version.group(1))


def _host_fresh(target) -> bool:
    return target is None or _fresh(target, [HOST_SRC, HEADER])


def up_to_date() -> bool:
    return _fresh(LIB, _deps()) and _host_fresh(_host_target())


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    return r


def _compile_host() -> str:
    torch = os.path.join(_torch_dir(), "include")
    obj = os.path.join(OBJ_DIR, "layers_host.cpp.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-I" + INCLUDE, "-isystem", torch, "-isystem",
          os.path.join(torch, "torch", "csrc", "api", "include"), "-isystem", cuda,
          "-I" + sysconfig.get_paths()["include"], "-c", HOST_SRC, "-o", obj], "g++ on " + HOST_SRC)
    return obj


def _link_host(obj: str, target: str) -> None:
    libs = os.path.join(_torch_dir(), "lib")
    tmp = target + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, "-L" + libs, "-ltorch_python", "-ltorch", "-ltorch_cpu",
          "-ltorch_cuda", "-lc10", "-lc10_cuda", "-L" + OUT_DIR, "-lgdr", "-Wl,-rpath," + libs,
          "-Wl,-rpath,$ORIGIN"], "link of " + target)
    os.replace(tmp, target)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    target = _host_target()
    library = force or not _fresh(LIB, _deps())
    host = target is not None and (force or not _host_fresh(target))
    os.makedirs(OUT_DIR, exist_ok=True)
    os.makedirs(OBJ_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        obj = ex.submit(_compile_host) if host else None
        if library:
            _build_library(verbose, extra_flags)
        if host:
            try:
                _link_host(obj.result(), target)
            except (OSError, RuntimeError) as e:
                warnings.warn(f"no compiled calls for the layers, they run from Python: {e}")
    return LIB


def _build_library(verbose, extra_flags) -> None:
    nvcc = _nvcc()
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

    with cf.ThreadPoolExecutor(max_workers=min(16, len(srcs))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs, "-ldl", "-lrt", "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
