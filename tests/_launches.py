"""The calls of the operators around the GEMMs over a recording stand-in for the CUDA runtime
(native/launch_recorder.cpp): what they ask of it, without a GPU."""
import ctypes
import os
import subprocess


def load(out_dir):
    from mxfp8_microscaled_precision_gb300 import build
    build.build()
    objs = [os.path.join(build.OUT, f + ".o") for f in ("api_block", "route", "permute", "norm", "clip")]
    if not all(map(os.path.exists, objs)):
        build.build(force=True)
    here = os.path.dirname(os.path.abspath(__file__))
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build._nvcc()))), "include")
    so = os.path.join(str(out_dir), "launch_recorder.so")
    r = subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-fPIC", "-shared", "-I" + cuda, "-I" + build.CSRC,
                        "-I" + build.INCLUDE, os.path.join(here, "native", "launch_recorder.cpp"), *objs, "-o", so,
                        "-Wl,-Bsymbolic"], capture_output=True, text=True)   # its own runtime, whatever else is loaded
    assert r.returncode == 0, r.stdout + r.stderr
    L = ctypes.CDLL(so, mode=ctypes.RTLD_LOCAL)
    L.rec_text.restype = ctypes.c_char_p
    L.rec_route.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int]
    L.rec_plan.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int]
    for f in (L.rec_norm, L.rec_norm_backward):
        f.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int64, ctypes.c_int64]
    L.rec_clip.argtypes = [ctypes.c_int, ctypes.c_int64, ctypes.c_int]
    return Recorder(L)


class Recorder:
    def __init__(self, L):
        self.L = L

    def __call__(self, call, *args, refuse=0, forget=True):
        """(status, launches, attributes): launches as (kernel, blocks, threads, shared bytes),
        attributes as (kernel, attribute, value); the launch number `refuse` (from 1 on) fails.  forget: an
        error that an earlier call left is dropped first."""
        self.L.rec_begin(refuse, 1 if forget else 0)
        status = getattr(self.L, "rec_" + call)(*args)
        launches, attributes = [], []
        for line in self.L.rec_text().decode().splitlines():
            kind, name, *numbers = line.split()
            if kind != "memset":
                (launches if kind == "launch" else attributes).append((name, *map(int, numbers)))
        return status, launches, attributes
