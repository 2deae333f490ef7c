"""Build libmuse_cores.so in-tree with nvcc for sm_100a, and the tensor front end of cores.py with g++.

    python -m gate_cores_b200.build [--force] [--verbose] [--jobs N]

Each .cu file compiles to its own object in parallel (the kernels share no
device symbols across files), then nvcc links the shared library.  The
library links the CUDA runtime statically, so it depends on the driver only;
the .so sits next to this file, where the binding looks for it.  The front end
(csrc/front.cpp) is a Python extension on PyTorch's headers that calls it.
"""
from __future__ import annotations

import argparse
import glob
import importlib.util
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
OBJ = os.path.join(ROOT, "_build", "muse_cores")
LIB = os.path.join(PKG, "libmuse_cores.so")
FRONT_SRC = os.path.join(CSRC, "front.cpp")
FRONT = os.path.join(PKG, "_front" + sysconfig.get_config_var("EXT_SUFFIX"))
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC,-O2,-Wall"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmuse_cores.so")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers() -> list[str]:
    return (glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
            glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(d) > t for d in sources() + _headers())


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")
    newest_dep = max(os.path.getmtime(d) for d in [src] + _headers())
    if os.path.exists(obj) and os.path.getmtime(obj) >= newest_dep:
        return obj
    tmp = obj + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, *FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", "-o", tmp, src]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, obj)
    return obj


def _without_front(why: str) -> None:
    # the C library is complete all the same; the calls that need the front end raise (an older one would not fit)
    if os.path.exists(FRONT):
        os.remove(FRONT)
    print(f"{os.path.basename(FRONT)} is not built: {why}", file=sys.stderr)


def _build_front(force: bool) -> None:
    spec = importlib.util.find_spec("torch")
    if spec is None:  # the C library is complete without it
        return
    torch = spec.submodule_search_locations[0]
    # (another PyTorch than the one it was built against: again)
    deps = [FRONT_SRC, os.path.join(torch, "version.py")] + glob.glob(os.path.join(INCLUDE, "*.h"))
    if not force and os.path.exists(FRONT) and all(os.path.getmtime(d) <= os.path.getmtime(FRONT) for d in deps):
        return
    if not os.path.exists(os.path.join(torch, "lib", "libtorch_cuda.so")):
        return _without_front("PyTorch is installed without CUDA")
    if shutil.which("g++") is None:
        return _without_front("there is no g++")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    headers = [INCLUDE, os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               cuda, sysconfig.get_paths()["include"]]
    tmp = FRONT + f".tmp{os.getpid()}"
    # g++, as nvcc takes it, whatever CXX is: the extension has to share PyTorch's libstdc++, and a compiler of another
    # make may link its own.  PyTorch's libraries are in the process before the extension is imported, so they need no
    # path here.
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
                           *(f for h in headers for f in ("-isystem" if h != INCLUDE else "-I", h)), FRONT_SRC, "-o", tmp,
                           "-L", PKG, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN",
                           "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10_cuda", "-lc10"])
    os.replace(tmp, FRONT)


def build(force: bool = False, verbose: bool = False, jobs: int | None = None) -> str:
    _build_lib(force, verbose, jobs)
    _build_front(force)
    return LIB


def _build_lib(force: bool, verbose: bool, jobs: int | None) -> None:
    if not force and not _stale():
        return
    os.makedirs(OBJ, exist_ok=True)
    if force:
        for o in glob.glob(os.path.join(OBJ, "*.o")):
            os.remove(o)
    srcs = sources()
    with ThreadPoolExecutor(max_workers=jobs or min(len(srcs), os.cpu_count() or 1)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([nvcc(), *ARCH, "-shared", "-o", tmp, *objs])
    os.replace(tmp, LIB)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--jobs", type=int, default=None)
    args = ap.parse_args()
    print(build(force=args.force, verbose=args.verbose, jobs=args.jobs))
