"""Sizes past a stated limit are refused before anything of that size is allocated."""
import pytest
import torch

from _util import gpu_or_skip

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gpu_or_skip()


@pytest.mark.parametrize("size", [33, 1025, 10 ** 6, 10 ** 8, 2 ** 31 - 1, 2 ** 40, 2 ** 62])
def test_a_refused_size_allocates_nothing(size):
    from mxfp8_microscaled_precision_gb300 import mxq
    x = torch.randn(4, 64, device="cuda")
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    calls = [lambda: mxq.route(x, size), lambda: mxq.route(x.bfloat16(), size)]
    if size > 1024:
        calls.append(lambda: mxq.moe_plan(ids, size))
    for call in calls:
        torch.cuda.synchronize()
        held = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        with pytest.raises(ValueError):
            call()
        assert torch.cuda.max_memory_allocated() - held <= 4096   # the small tensors that the test makes itself
