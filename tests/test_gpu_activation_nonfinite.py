"""NaN and infinities in the activation's input, forward: each shows in its own place of the output and nowhere else."""
import pytest
import torch

from _util import gpu_or_skip

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("keep", [True, False], ids=["kept", "not_kept"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
@pytest.mark.parametrize("inter", [96, 100], ids=["vectors", "any"])
def test_forward_results_of_nan_and_infinities(inter, gated, kind, dtype, keep):
    """f(inf) = inf; f(-inf) is minus infinity times zero, NaN, as the formula has it; a product with u as IEEE has it."""
    gpu_or_skip()
    from mxfp8_microscaled_precision_gb300 import mxq
    gen = torch.Generator().manual_seed(1)
    z = torch.randn(6, inter * (2 if gated else 1), generator=gen).to(dtype).cuda()
    clean = mxq.activation(z, kind=kind, gated=gated, checkpoint=keep)[0]
    want = clean.clone()
    for row, col, value, result in ((1, 3, NAN, NAN), (2, 40, INF, INF), (3, 95, -INF, NAN), (4, 31, -NAN, NAN)):
        z[row, col] = value
        if gated and result == INF:
            result = result if float(z[row, inter + col]) > 0 else -INF
        want[row, col] = result
    if gated:
        g = float(z[5, 8])
        z[5, inter + 8], z[0, inter + 50] = -INF, NAN
        want[5, 8], want[0, 50] = (-INF if g > 0 else INF), NAN
    y = mxq.activation(z, kind=kind, gated=gated, checkpoint=keep)[0]
    hit = want.isnan()
    assert int(hit.sum()) == (4 if gated else 3)
    assert torch.equal(y.isnan(), hit)
    assert torch.equal(y[~hit], want[~hit])
    assert int(y.isinf().sum()) == (2 if gated else 1)
