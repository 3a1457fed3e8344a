"""The mixture-of-experts block of examples/moe_block.py with its activation kept in 8 bits, and with its experts in
4 bits, on the GPU.

Tolerances (2-norms).  Training: a product's operands in E4M3 put a gradient behind four of them off by 0.10
(2^-4 / sqrt 3 = 0.036 a value, sqrt 2 of it a product); the activation's input, kept with the same error, enters dz once more,
in f' and in u, so by up to sqrt 2 0.036 = 0.051: together 0.112, half as much again 0.17.
Decoding: the reference quantizes the same way in 64 bits; what is left are roundings to BF16 (three on the way, 2^-9 each
in the mean) and values that such a rounding moves to the other side of an E2M1 border: a value lies within 2^-9 of itself of
one with probability 2^-7 at most (the borders are a quarter apart at least) and moves by up to a third of itself then,
sqrt(2^-7) / 3 = 0.03; with half as much again 0.045."""
import os
import sys

import numpy as np
import pytest
import torch

import _fp4
from _util import gpu_or_skip
from test_gpu_moe_block import _off, _reference

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gpu_or_skip()


@pytest.mark.parametrize("T,masked", [(1, False), (300, True), (513, False)])
def test_training_with_the_activation_in_8_bits(T, masked):
    from mxfp8_microscaled_precision_gb300 import mxq, workloads
    import moe_block
    block = moe_block.MoEBlock(256, 128, 8, 2, seed=3, checkpoint8=True)
    block.router *= 20
    x, dout = workloads.normal((T, 256), 1.0, 11, device="cuda"), workloads.normal((T, 256), 1.0, 12, device="cuda")
    mask = torch.rand(T, generator=torch.Generator().manual_seed(1)).cuda() > 0.2 if masked else None
    out, saved = block.forward(x, token_mask=mask)
    assert saved[11] is None and [t.dtype for t in saved[10]] == [torch.uint8, torch.uint8]
    ref, dx_ref, grads_ref = _reference(block, x, saved[5], dout, mask)
    assert _off(mxq.moe_combine(saved[12], saved[8], saved[6]), ref - x.double()) < 0.11 + 2.0 ** -8
    dx, grads = block.backward(dout, saved)
    share = float((dx_ref - dout.double()).norm() / dx_ref.norm())
    assert _off(dx, dx_ref) < 2.0 ** -8 + (0.17 + 2.0 ** -8) * share
    for name, g, r in zip(("norm_w", "norm_b", "router", "gate_up", "down"), grads, grads_ref):
        assert torch.isfinite(g).all() and _off(g, r) < 0.17, (name, _off(g, r))
    assert mxq.get_device_status() == 0


def _held(x):
    codes, scales = _fp4.quantize(x, "e2m1")
    return _fp4.values(codes, scales, x.shape[1], "e2m1")


@pytest.mark.parametrize("T,masked", [(1, False), (5, False), (64, True), (400, False)])
def test_decoding_through_weights_in_4_bits(T, masked):
    from mxfp8_microscaled_precision_gb300 import mxq, workloads
    import moe_block
    block = moe_block.MoEBlock(256, 96, 8, 2, seed=3)
    block.router *= 20
    block.quantize_for_serving()
    x = workloads.normal((T, 256), 1.0, 11, device="cuda")
    mask = torch.rand(T, generator=torch.Generator().manual_seed(1)).cuda() > 0.2 if masked else None
    out = block.decode(x, token_mask=mask)
    h, _, _ = mxq.layer_norm(x, block.norm_w, block.norm_b)
    ids, w = mxq.route(h.float() @ block.router.t(), 2, score="sigmoid", bias=block.bias, token_mask=mask)
    h, ids, w = _held(_fp4.f64(h)), ids.cpu().numpy(), _fp4.f64(w)
    share = np.zeros((T, 256))
    for e in range(8):
        gu, dn = _held(_fp4.f64(block.w_gate_up[e])), _held(_fp4.f64(block.w_down[e]))
        for j in range(2):
            t = np.nonzero(ids[:, j] == e)[0]
            if len(t):
                z = h[t] @ gu.T
                act = z[:, :96] / (1 + np.exp(-z[:, :96])) * z[:, 96:]
                share[t] += w[t, j:j + 1] * (_held(act) @ dn.T)
    if masked:
        assert torch.equal(out[~mask], x[~mask])
    got = _fp4.f64(out) - _fp4.f64(x)
    # the sum with x is rounded to BF16, by half a step of the sum
    rounding = 2.0 ** -9 * np.linalg.norm(_fp4.f64(x))
    assert np.linalg.norm(got - share) < 0.045 * np.linalg.norm(share) + rounding
    assert mxq.get_device_status() == 0


def test_a_step_of_the_example_runs():
    import moe_block
    from mxfp8_microscaled_precision_gb300 import workloads
    block = moe_block.MoEBlock(256, 128, 8, 2, checkpoint8=True)
    x = workloads.normal((200, 256), 1.0, 7, device="cuda")
    loss, norm = block.step(x, x * 0.5)
    assert torch.isfinite(loss) and torch.isfinite(norm)
