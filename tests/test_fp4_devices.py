"""Devices of the tensors of one call (MXFP4, and activations kept in 8 bits).  Stand-ins that say they live on a GPU and
have no memory take the place of tensors: a call refuses them before it touches anything."""
import pytest
import torch

from _util import gpu_or_skip
from test_block_devices import StandIn

B, F, I64, U8 = torch.bfloat16, torch.float32, torch.int64, torch.uint8
M, N, K, G = 4, 16, 64, 2
ATOM = 512


def _calls():
    """{name: (call of its tensors, [(shape, dtype) of each])}"""
    from mxfp8_microscaled_precision_gb300 import mxq
    x, q, s = ((M, K), B), ((M, K // 2), U8), ((ATOM,), U8)
    grouped, off = (((1 + G) * ATOM,), U8), ((G + 1,), I64)
    act, kept, scales = ((M, K // 2), B), ((M, K), U8), ((M, 2), U8)
    return {
        "quant": (lambda x, a, b, c, d: mxq.quant_mxfp4(x, out=(a, b, c, d)), [x, q, s, ((K, 16), U8), s]),
        "quant_grouped": (lambda x, o, q, s: mxq.quant_mxfp4_grouped(x, o, out=(q, s)), [x, off, q, grouped]),
        "dequant": (lambda q, s, o: mxq.dequant_1x32(q, s, K, fmt="e2m1", out=o), [q, s, x]),
        "dequant_plain": (lambda q, s, o: mxq.dequant_1x32(q, s, K, layout="rowmajor", out=o), [kept, scales, x]),
        "gemm": (lambda a, s, b, t, y: mxq.gemm_mxfp4(a, s, b, t, M, N, K, out=y), [q, s, ((N, K // 2), U8), s, ((M, N), B)]),
        "grouped_gemm": (lambda a, s, b, t, o, y: mxq.grouped_gemm_mxfp4(a, s, b, t, o, N, K, out=y),
                         [q, grouped, ((G * N, K // 2), U8), ((G * ATOM,), U8), off, ((M, N), B)]),
        "quant_cols_grouped": (lambda x, o, q, s: mxq.quant_mxfp4_cols_grouped(x, o, out=(q, s)),
                               [x, off, ((K, 64 * (1 + G)), U8), (((1 + G) * ATOM,), U8)]),
        "wgrad": (lambda a, s, b, t, o, y: mxq.grouped_gemm_mxfp4_wgrad(a, s, b, t, o, M, out=y),
                  [((N, 64 * (1 + G)), U8), grouped, ((K, 64 * (1 + G)), U8), grouped, off, ((G, N, K), B)]),
        "activation": (lambda z, y, q, s: mxq.activation(z, out=(y, q, s)), [x, act, kept, scales]),
        "activation_backward": (lambda d, q, s, z, y: mxq.activation_backward(d, q, s, out=(z, y)), [act, kept, scales, x, act]),
    }


NAMES = ["quant", "quant_grouped", "quant_cols_grouped", "wgrad", "dequant", "dequant_plain", "gemm", "grouped_gemm", "activation", "activation_backward"]


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_two_devices_are_refused(name):
    from mxfp8_microscaled_precision_gb300 import build
    build.build()
    call, shapes = _calls()[name]
    for odd in range(len(shapes)):
        with pytest.raises(ValueError, match="cuda:1.*cuda:0|cuda:0.*cuda:1"):
            call(*[StandIn(*s, 1 if i == odd else 0) for i, s in enumerate(shapes)])


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_another_device_than_the_current_one_are_refused(name):
    gpu_or_skip()
    current = torch.cuda.current_device()
    call, shapes = _calls()[name]
    with pytest.raises(ValueError, match="current device"):
        call(*[StandIn(*s, current + 1) for s in shapes])
