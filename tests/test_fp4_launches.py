"""What MXFP4 quantization, a payload's values and the activation ask of the CUDA runtime (no GPU needed): a recording
stand-in takes its place."""
import ctypes
import os
import subprocess

import pytest

import _launches

MAX_DYNAMIC = 8            # cudaFuncAttributeMaxDynamicSharedMemorySize
BLOCK_BYTES = 227 * 1024   # shared memory of a block at most
BF16, F32 = 0, 1


@pytest.fixture(scope="module")
def record(tmp_path_factory):
    from mxfp8_microscaled_precision_gb300 import build
    build.build()
    objs = [os.path.join(build.OUT, f + ".o") for f in ("api_block", "route", "permute", "norm", "clip", "api_fp4", "fp4", "act")]
    if not all(map(os.path.exists, objs)):
        build.build(force=True)
    here = os.path.dirname(os.path.abspath(__file__))
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build._nvcc()))), "include")
    so = os.path.join(str(tmp_path_factory.mktemp("recorder")), "fp4_recorder.so")
    r = subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-fPIC", "-shared", "-I" + cuda, "-I" + build.CSRC,
                        "-I" + build.INCLUDE, os.path.join(here, "native", "fp4_recorder.cpp"), *objs, "-o", so, "-Wl,-Bsymbolic"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    L = ctypes.CDLL(so, mode=ctypes.RTLD_LOCAL)
    L.rec_text.restype = ctypes.c_char_p
    I32, I64 = ctypes.c_int, ctypes.c_int64
    L.rec_quant4.argtypes = [I32, I64, I64, I64, I32]
    L.rec_quant4_grouped.argtypes = [I32, I64, I64, I32, I32]
    L.rec_values.argtypes = [I32, I32, I64, I64]
    L.rec_act.argtypes = [I32, I64, I64, I32]
    return _launches.Recorder(L)


@pytest.mark.parametrize("sms", [152, 148, 100, 76])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_few_rows_are_those_that_one_wave_of_this_device_holds(record, sms, dtype):
    """Blocks of eight rows as long as there are at most eight for each SM that the device has, whatever their shape."""
    record.L.rec_sms(sms)
    tall = 128 // (2 << dtype)
    for cols, across in ((256, 1), (200, 1), (4096, 16)):
        for batch in (1, 2):
            most = 8 * sms // (across * batch)   # blocks down a matrix
            few = record("quant4", dtype, batch, 8 * most, cols, 1)[1]
            assert [n[1] for n in few] == [most * across * batch]
            rows = 8 * most + 1
            many = record("quant4", dtype, batch, rows, cols, 1)[1]
            assert [n[1] for n in many] == [-(-rows // 128) * (128 // tall) * across * batch]
    record.L.rec_sms(152)


@pytest.mark.parametrize("sms", [152, 148, 100, 76])
@pytest.mark.parametrize("copies", [2, 3])
def test_few_fp32_tiles_are_two_for_each_sm_of_this_device(record, sms, copies):
    record.L.rec_sms(sms)
    for tiles, threads in ((1, 512), (2 * sms, 512), (2 * sms + 1, 256)):
        launched = record("quant4", F32, 1, 128 * tiles, 128, copies)[1]
        assert [(n[1], n[2]) for n in launched] == [(tiles, threads)]
        assert [n[2] for n in record("quant4", BF16, 1, 128 * tiles, 128, copies)[1]] == [256]
    record.L.rec_sms(152)


CALLS = ([("quant4", (d, b, r, c, k)) for d in (BF16, F32) for b, r, c in ((1, 8, 4096), (3, 300, 77), (1, 4096, 7168)) for k in (1, 2, 3)]
         + [("quant4_grouped", (d, r, c, 5, k)) for d in (BF16, F32) for r, c in ((9, 96), (4096, 1111)) for k in (0, 1)]
         + [("values", (d, e, r, c)) for d in (BF16, F32) for e in (0, 1, 2) for r, c in ((5, 64), (1000, 1111))]
         + [("act", (d, r, i, k)) for d in (BF16, F32) for r, i in ((64, 2048), (4099, 1111)) for k in (0, 1)])


@pytest.mark.parametrize("call,args", CALLS, ids=str)
def test_a_refused_launch_is_reported_and_leaves_no_error_behind(record, call, args):
    status, launches, attributes = record(call, *args)
    assert status == 0 and len(launches) == 1
    kernel, blocks, threads, shared = launches[0]
    assert blocks >= 1 and 1 <= threads <= 1024 and shared <= BLOCK_BYTES
    if shared > 48 * 1024:
        assert (kernel, MAX_DYNAMIC, shared) in attributes
    status, done, _ = record(call, *args, refuse=1)
    assert status != 0 and done == []
    assert record("route", 100, 64, 4, forget=False)[0] == 0


def test_a_kernels_shared_memory_limit_does_not_depend_on_the_shape(record):
    limits = {}
    for call, args in CALLS:
        for kernel, attribute, value in record(call, *args)[2]:
            if attribute == MAX_DYNAMIC:
                limits.setdefault(kernel, set()).add(value)
    assert limits and all(len(v) == 1 for v in limits.values())
