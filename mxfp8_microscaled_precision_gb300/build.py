"""Build libmxq.so (the CUDA library) in-tree with nvcc for sm_103a, and the
extension module that calls it from Python (csrc/calls.cpp) with g++.

The translation units are compiled in parallel, then linked into
``mxfp8_microscaled_precision_gb300/_build/libmxq.so`` (the CUDA runtime is
linked statically, the driver API is reached through the runtime's entry
point query, so the library needs nothing but the NVIDIA driver at run time).
"""
from __future__ import annotations

import concurrent.futures as cf
import fcntl
import functools
import importlib.util
import os
import re
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT = os.path.join(PKG, "_build")
LIB = os.path.join(OUT, "libmxq.so")
SOURCES = ["api.cu", "quant.cu", "gemm.cu", "tensor_map.cu", "fsdp.cu", "noalloc.cu",
           "api_block.cu", "route.cu", "permute.cu", "norm.cu", "clip.cu"]
HEADERS = ["mxq_device.cuh", "mxq_internal.h", "mxq_quant_math.cuh", "mxq_elem.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I" + INCLUDE, "-I" + CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: set NVCC or put the CUDA toolkit on PATH")


def _torch_dir() -> str:
    return os.path.dirname(importlib.util.find_spec("torch").origin)


@functools.lru_cache(maxsize=None)
def _torch_version() -> str:
    """Of the torch that would be imported, without importing it."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return re.search(r"""^__version__\s*=\s*['"]([^'"]+)""", f.read(), re.MULTILINE).group(1)


def calls_path() -> str:
    """The extension module, by the Python and the torch that it is built for: torch's C++
    interface is not the same from one version to the next."""
    return os.path.join(OUT, f"_mxqcall-torch-{_torch_version()}" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(calls_path()):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(calls_path()))
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS + ["calls.cpp"]] + [os.path.join(INCLUDE, "mxq.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (if needed) and return the path of libmxq.so.  Processes that
    build at the same time (one per rank) take turns on a lock file."""
    if not force and not _stale():
        return LIB
    os.makedirs(OUT, exist_ok=True)
    with open(os.path.join(OUT, ".build.lock"), "w") as lock:
        fcntl.flock(lock, fcntl.LOCK_EX)
        try:
            if not force and not _stale():   # another process built it meanwhile
                return LIB
            return _build(verbose)
        finally:
            fcntl.flock(lock, fcntl.LOCK_UN)


def _gxx() -> str:
    return os.environ.get("CXX", "g++")


def _compile_calls() -> str:
    obj = os.path.join(OUT, "calls.o")
    include = os.path.join(_torch_dir(), "include")
    r = subprocess.run([_gxx(), "-O2", "-std=c++17", "-Wall", "-fPIC", "-I" + INCLUDE,
                        "-I" + sysconfig.get_paths()["include"], "-isystem", include, "-isystem",
                        os.path.join(include, "torch", "csrc", "api", "include"), "-c", os.path.join(CSRC, "calls.cpp"),
                        "-o", obj], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for calls.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _build(verbose: bool) -> str:
    nvcc = _nvcc()
    objs = []

    def compile_one(src):
        obj = os.path.join(OUT, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        calls = ex.submit(_compile_calls)
        objs = list(ex.map(compile_one, SOURCES))
        calls_obj = calls.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    # torch's libraries are in the process before the module is: no path to them is needed
    calls_so = calls_path()
    tmp = calls_so + f".tmp{os.getpid()}"
    r = subprocess.run([_gxx(), "-shared", "-o", tmp, calls_obj, "-L" + OUT, "-l:libmxq.so", "-Wl,-rpath,$ORIGIN",
                        "-L" + os.path.join(_torch_dir(), "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10"],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed for calls.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, calls_so)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
