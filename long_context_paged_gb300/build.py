"""Build the CUDA library ``_lib/libpagedattn.so`` in-tree with nvcc (sm_103a only).

Each ``csrc/*.cu`` translation unit is compiled to an object in parallel, then linked into
one shared library that exports the C ABI declared in ``include/pagedattn.h``. Beside it,
``_lib/_pa_call.so`` is the Python binding's fast path (``csrc/fastcall.cpp``, host C++ against the
installed PyTorch's headers). The binding does without it where it cannot be built.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIB_DIR, "libpagedattn.so")
INCLUDE = os.path.join(ROOT, "include")
FAST_SRC = os.path.join(CSRC, "fastcall.cpp")
FAST = os.path.join(LIB_DIR, "_pa_call.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
                     "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _build_fast(verbose: bool, force: bool):
    """Compile the binding's fast path; returns its error text, or None. Rebuilt when its source, the
    C ABI or the installed PyTorch changed."""
    try:
        import torch
    except ImportError as e:
        return f"PyTorch cannot be imported ({e})"
    stamp = os.path.join(BUILD, "_pa_call.torch")
    known = open(stamp).read() if os.path.exists(stamp) else ""
    if not force and known == torch.__version__ and not _stale(FAST, [FAST_SRC, __file__] + _headers()):
        return None
    if os.path.exists(FAST):
        os.remove(FAST)
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = FAST + ".tmp"
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-fPIC", "-shared", "-std=c++17", "-I", INCLUDE,
           "-I", os.path.join(base, "include"),
           "-I", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", FAST_SRC, "-o", tmp,
           "-L", LIB_DIR, "-lpagedattn", "-L", os.path.join(base, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        return str(e)
    if r.returncode != 0:
        return r.stderr[-2000:]
    os.replace(tmp, FAST)
    with open(stamp, "w") as f:
        f.write(torch.__version__)
    return None


def build(verbose: bool = False, force: bool = False, extra_flags=()) -> str:
    """Compile and link the library if any source changed; returns the library path."""
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    cc = nvcc()
    headers = _headers()
    jobs = []
    objs = []
    for src in _sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src, __file__] + headers):
            jobs.append([cc, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj])

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed ({os.path.basename(cmd[-3])}):\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)

    if jobs:
        with ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            list(ex.map(run, jobs))
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + ".tmp"
        run([cc, *ARCH, "-shared", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    error = _build_fast(verbose, force)
    if error is not None:
        print(f"the binding's fast path was not built, calls take its slower one: {error}",
              file=sys.stderr)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
