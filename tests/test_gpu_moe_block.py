"""The mixture-of-experts block of examples/moe_block.py on the GPU, forward and
backward, against the same block in 64 bits without quantization.

Tolerance: E4M3 keeps 3 bits after the leading one and rounds to nearest, an error
that is even over +-2^-4 of a value at most: 2^-4 / sqrt(3) = 0.036 in the mean square.  A product of two
quantized operands is off by sqrt(2) 0.036 = 0.051 of its size (the terms' errors are
independent), so a result behind two products by 0.072 and a gradient behind four
by 0.10; the bounds are half as much again, 0.11 and 0.15 (2-norms).  What lies before the
first product (the choice, the plan) is exact or FP32.  out and dx also hold x and dout, next to
which the block's own share is small: a result in BF16 is rounded by at most 2^-8 of itself."""
import os
import sys

import pytest
import torch

from _util import gpu_or_skip

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gpu_or_skip()


def _reference(block, x, ids, dout, mask):
    """out and gradients in 64 bits by autograd, with the given choice of experts."""
    ps = [p.detach().double().requires_grad_() for p in block.parameters()]
    nw, nb, router, wgu, wd = ps
    xd = x.double().requires_grad_()
    mu = xd.mean(1, keepdim=True)
    h = (xd - mu) / torch.sqrt(((xd - mu) ** 2).mean(1, keepdim=True) + 1e-5) * nw + nb
    s = torch.sigmoid(h @ router.t())
    keep = (ids >= 0).double()
    chosen = s.gather(1, ids.long().clamp(min=0)) * keep
    w = chosen / (chosen.sum(1, keepdim=True) + 1e-20)
    out = xd
    for j in range(ids.shape[1]):
        for e in range(block.E):
            t = torch.nonzero(ids[:, j] == e)[:, 0]
            if len(t) == 0:
                continue
            z = h[t] @ wgu[e].t()
            y = (torch.nn.functional.silu(z[:, :block.I]) * z[:, block.I:]) @ wd[e].t()
            out = out.index_add(0, t, y * w[t, j:j + 1])
    (out * dout.double()).sum().backward()
    return out.detach(), xd.grad, [p.grad for p in ps]


def _off(got, want):
    d = want.double()
    return float((got.double() - d).norm() / d.norm())


@pytest.mark.parametrize("T,masked", [(1, False), (7, False), (300, True), (513, False)])
def test_block_forward_and_backward(T, masked):
    from mxfp8_microscaled_precision_gb300 import mxq, workloads
    import moe_block
    block = moe_block.MoEBlock(256, 128, 8, 2, seed=3)
    block.router *= 20
    x = workloads.normal((T, 256), 1.0, 11, device="cuda")
    dout = workloads.normal((T, 256), 1.0, 12, device="cuda")
    mask = None
    if masked:
        mask = torch.rand(T, generator=torch.Generator().manual_seed(1)).cuda() > 0.2
    out, saved = block.forward(x, token_mask=mask)
    ids, offsets = saved[5], saved[7]
    if masked:
        assert (ids[~mask] == -1).all() and torch.equal(out[~mask], x[~mask])
    assert int(offsets[-1]) == int((ids >= 0).sum())
    ref, dx_ref, grads_ref = _reference(block, x, ids, dout, mask)
    share = float((ref - x.double()).norm() / ref.norm())
    assert _off(out, ref) < 2.0 ** -8 + (0.11 + 2.0 ** -8) * share
    assert _off(mxq.moe_combine(saved[12], saved[8], saved[6]), ref - x.double()) < 0.11 + 2.0 ** -8
    dx, grads = block.backward(dout, saved)
    share = float((dx_ref - dout.double()).norm() / dx_ref.norm())
    assert _off(dx, dx_ref) < 2.0 ** -8 + (0.15 + 2.0 ** -8) * share
    for name, g, r in zip(("norm_w", "norm_b", "router", "gate_up", "down"), grads, grads_ref):
        assert torch.isfinite(g).all() and _off(g, r) < 0.15, (name, _off(g, r))
    assert mxq.get_device_status() == 0
