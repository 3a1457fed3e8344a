"""Buffers that a caller gives to mxq.layer_norm, and rows without a column."""
import pytest
import torch

from _util import gpu_or_skip

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gpu_or_skip()


@pytest.mark.parametrize("C", [64, 97])
@pytest.mark.parametrize("given", [(0,), (1,), (2,), (0, 1), (0, 2), (1, 2), (0, 1, 2)])
def test_every_buffer_that_is_given_is_written_and_returned(C, given):
    from mxfp8_microscaled_precision_gb300 import mxq
    x = torch.randn(9, C, device="cuda").bfloat16()
    want = mxq.layer_norm(x)
    out = [torch.full_like(w, 7.0) if i in given else None for i, w in enumerate(want)]
    got = mxq.layer_norm(x, out=out)
    for i, w in enumerate(want):
        assert torch.equal(got[i], w)
        if i in given:
            assert got[i] is out[i] and torch.equal(out[i], w)


def test_a_statistic_that_does_not_fit_is_refused():
    from mxfp8_microscaled_precision_gb300 import mxq
    x = torch.randn(9, 64, device="cuda")
    good = torch.empty(9, device="cuda")
    for bad in (good.double(), good[:8], good.cpu(), torch.empty(18, device="cuda")[::2]):
        for out in ((None, bad, None), (None, None, bad), (None, good, bad), (None, bad, good)):
            with pytest.raises(ValueError):
                mxq.layer_norm(x, out=out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_statistics_of_rows_without_a_column(dtype):
    """0 / 0: NaN in every row, and not what the memory held."""
    from mxfp8_microscaled_precision_gb300 import mxq
    x = torch.empty(5, 0, dtype=dtype, device="cuda")
    mean, rstd = (torch.full((5,), 7.0, device="cuda") for _ in range(2))
    y, m, r = mxq.layer_norm(x, out=(None, mean, rstd))
    assert y.shape == (5, 0) and m is mean and r is rstd
    assert torch.isnan(mean).all() and torch.isnan(rstd).all()
    dx, dw, db = mxq.layer_norm_backward(x, x, None, mean, rstd)
    assert dx.shape == (5, 0) and dw.shape == db.shape == (0,)
