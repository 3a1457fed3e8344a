"""The scale of routing weights and their gradient on the GPU (mxq.route_backward)."""
import pytest
import torch

from _util import gpu_or_skip

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gpu_or_skip()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("scale", [1.0, 2.5, 0.3, 1.7, 1e-3, -2.9])
def test_one_expert_with_all_the_weight_has_no_gradient_at_any_scale(score, scale, dtype):
    """top 1, renormalised: the weight is the scale whatever the logits are.  s / s is 1 and dw - dw is 0, whatever
    the scale rounds."""
    from mxfp8_microscaled_precision_gb300 import mxq
    gen = torch.Generator(device="cuda").manual_seed(11)
    for E in (5, 72, 128, 360, 1024):
        x = (3.0 * torch.randn(1000, E, generator=gen, device="cuda")).to(dtype)
        dw = torch.randn(1000, 1, generator=gen, device="cuda")
        ids, _ = mxq.route(x, 1, score=score, renorm=True, scale=scale)
        assert (mxq.route_backward(dw, x, ids, score=score, renorm=True, scale=scale) == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_scale_of_two_doubles_every_bit_pattern(score):
    from mxfp8_microscaled_precision_gb300 import mxq
    gen = torch.Generator(device="cuda").manual_seed(12)
    x = torch.randn(500, 100, generator=gen, device="cuda")
    dw = torch.randn(500, 6, generator=gen, device="cuda")
    ids, _ = mxq.route(x, 6, score=score)
    one, two = (mxq.route_backward(dw, x, ids, score=score, scale=s) for s in (1.0, 2.0))
    assert torch.equal(2 * one, two)
