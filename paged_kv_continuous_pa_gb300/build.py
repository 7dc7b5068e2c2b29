"""Build libpa_gb300.so in-tree with nvcc for sm_103a.

Each .cu under csrc/ compiles to an object in parallel, then one nvcc link
produces ``_lib/libpa_gb300.so``.  Rebuilds only what changed (object newer
than its source and every header).  Beside it ``_lib/pa_bind.so``, the binding's
short way into the library, is compiled with g++ against the installed torch; the library
needs neither, and is built without it where there is no torch.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
OBJ_DIR = os.path.join(HERE, "_build")
LIB_DIR = os.path.join(HERE, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libpa_gb300.so")
BIND_SOURCE = os.path.join(CSRC, "pa_bind.cpp")
BIND_PATH = os.path.join(LIB_DIR, "pa_bind.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", f"-I{INCLUDE}"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (CUDA toolkit required to build libpa_gb300)")


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build_bind(force: bool = False) -> str:
    """Compile the extension module pa_bind (host code; g++, torch's headers and libraries)."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    if not force and not _stale(BIND_PATH, [BIND_SOURCE, os.path.join(INCLUDE, "pa.h"), torch.__file__]):
        return BIND_PATH
    os.makedirs(LIB_DIR, exist_ok=True)
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    tmp = BIND_PATH + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-fPIC", "-shared", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{sysconfig.get_paths()['include']}",
           f"-I{cuda}"] + [f"-I{p}" for p in cpp_extension.include_paths()] + \
          [BIND_SOURCE, "-o", tmp, f"-L{lib}", f"-Wl,-rpath,{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on pa_bind.cpp:\n{r.stdout}\n{r.stderr[-4000:]}")
    os.replace(tmp, BIND_PATH)
    return BIND_PATH


def build(force: bool = False, verbose: bool = False, extra_flags=(), variant: str = "") -> str:
    """Compile and link; returns the library path.  A non-empty `variant` builds
    a separately named library (objects under _build/<variant>/) with
    `extra_flags`, e.g. a tuning constant overridden with -D, leaving the
    default library untouched."""
    obj_dir = os.path.join(OBJ_DIR, variant) if variant else OBJ_DIR
    lib_path = os.path.join(LIB_DIR, f"libpa_gb300_{variant}.so") if variant else LIB_PATH
    os.makedirs(obj_dir, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    heads = _headers()
    cc = nvcc()
    jobs = []
    objs = []
    for s in srcs:
        o = os.path.join(obj_dir, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if force or _stale(o, [s] + heads):
            jobs.append((s, o))

    def compile_one(job):
        s, o = job
        tmp = o + f".tmp{os.getpid()}"
        cmd = [cc] + ARCH + NVCC_FLAGS + list(extra_flags) + ["-c", s, "-o", tmp]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(s)}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        os.replace(tmp, o)

    def bind_beside():
        if variant or importlib.util.find_spec("torch") is None:
            return
        try:
            build_bind(force)
        except Exception as e:  # the calls go through ctypes without it
            if os.path.exists(BIND_PATH):  # one of older sources
                os.remove(BIND_PATH)
            warnings.warn(f"pa_bind was not built: {e}", RuntimeWarning)

    with cf.ThreadPoolExecutor(max(1, min(len(jobs) + 1, os.cpu_count() or 4))) as ex:
        bind = ex.submit(bind_beside)
        list(ex.map(compile_one, jobs))
        bind.result()
    if force or jobs or _stale(lib_path, objs):
        tmp = lib_path + f".tmp{os.getpid()}"
        cmd = [cc] + ARCH + ["-shared", "-o", tmp] + objs + ["-Xcompiler", "-fPIC"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, lib_path)
    return lib_path


if __name__ == "__main__":  # pragma: no cover
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
