"""Devices of the tensors of one call (mxq's operators around the GEMMs).  Stand-ins that say they live on a GPU
and have no memory take the place of tensors: a call refuses them before it touches anything."""
import pytest
import torch

from _util import gpu_or_skip


class StandIn(torch.Tensor):
    @staticmethod
    def __new__(cls, shape, dtype, index):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device=f"cuda:{index}")

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise AssertionError(f"{func} of a stand-in")


B, F, I32, I64, U8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8
T, E, K, H = 4, 8, 2, 16


def _calls():
    """{name: (call of its tensors, [(shape, dtype) of each])}"""
    from mxfp8_microscaled_precision_gb300 import mxq
    rows, tokens, slots, weights = ((T * K, H), B), ((T, H), B), ((T, K), I32), ((T, K), F)
    row, stat = ((H,), F), ((T,), F)
    return {
        "route": (lambda x, b, m, i, w: mxq.route(x, K, bias=b, token_mask=m, out=(i, w)),
                  [((T, E), F), ((E,), F), ((T,), U8), slots, weights]),
        "route_backward": (lambda d, x, i, o: mxq.route_backward(d, x, i, out=o), [weights, ((T, E), F), slots, ((T, E), F)]),
        "plan": (lambda i, o, r: mxq.moe_plan(i, E, out=(o, r)), [slots, ((E + 1,), I64), slots]),
        "dispatch": (lambda x, r, a: mxq.moe_dispatch(x, r, out=a), [tokens, slots, rows]),
        "combine": (lambda y, r, w, o: mxq.moe_combine(y, r, w, out=o), [rows, slots, weights, tokens]),
        "combine_backward": (lambda d, y, r, w, a, b: mxq.moe_combine_backward(d, y, r, w, out=(a, b)),
                             [tokens, rows, slots, weights, rows, weights]),
        "layer_norm": (lambda x, w, s, y, m, r: mxq.layer_norm(x, w, s, out=(y, m, r)), [tokens, row, row, tokens, stat, stat]),
        "layer_norm_backward": (lambda d, x, w, m, r, o: mxq.layer_norm_backward(d, x, w, m, r, out=o),
                                [tokens, tokens, row, stat, stat, tokens]),
        "grad_norm": (lambda *g: mxq.grad_norm(g), [row, tokens, row]),
        "clip": (lambda a, b, c, d: mxq.clip_grad_norm([a, b], 1.0, out=[c, d]), [row, tokens, row, tokens]),
    }


NAMES = ["route", "route_backward", "plan", "dispatch", "combine", "combine_backward", "layer_norm", "layer_norm_backward",
         "grad_norm", "clip"]


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_two_devices_are_refused(name):
    from mxfp8_microscaled_precision_gb300 import build
    build.build()
    call, shapes = _calls()[name]
    for odd in range(len(shapes)):
        with pytest.raises(ValueError, match="cuda:1.*cuda:0|cuda:0.*cuda:1"):
            call(*[StandIn(*s, 1 if i == odd else 0) for i, s in enumerate(shapes)])


@pytest.mark.gpu
@pytest.mark.parametrize("name", [n for n in NAMES if n not in ("layer_norm_backward", "grad_norm", "clip")])
def test_tensors_of_another_device_than_the_current_one_are_refused(name):
    """The calls whose results can all be given: the others allocate some on that device first."""
    gpu_or_skip()
    current = torch.cuda.current_device()
    call, shapes = _calls()[name]
    with pytest.raises(ValueError, match="current device"):
        call(*[StandIn(*s, current + 1) for s in shapes])
