"""A contraction so long that one tile takes seconds: the bounded waits of the products allow for it."""
import pytest
import torch

from _util import gpu_or_skip

pytestmark = pytest.mark.gpu


def test_weight_gradient_of_one_column_over_nearly_all_rows_there_can_be():
    """2^31 - 8192 rows of one expert, some 8.4 million pipeline stages of a single tile.  The first and the last 40 rows are
    ones and the others zero: the sum is 80, exactly."""
    gpu_or_skip()
    from mxfp8_microscaled_precision_gb300 import mxq
    if torch.cuda.mem_get_info()[0] < 32 << 30:
        pytest.skip("needs 32 GB")
    R = 2 ** 31 - 8192
    x = torch.zeros(R, 1, dtype=torch.bfloat16, device="cuda")
    x[:40] = 1
    x[-40:] = 1
    off = torch.tensor([0, R], device="cuda")
    q, s = mxq.quant_mxfp4_cols_grouped(x, off)
    y = mxq.grouped_gemm_mxfp4_wgrad(q, s, q, s, off, R)
    assert mxq.get_device_status() == 0
    assert y.shape == (1, 1, 1) and float(y) == 80.0
    del x, q, s
    torch.cuda.empty_cache()
