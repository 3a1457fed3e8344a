"""Experts' offsets that break the rule: the MXFP4 calls leave rows unspecified and stay inside their buffers and
launches."""
import pytest
import torch

from _util import gpu_or_skip

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gpu_or_skip()


# The launch holds (min(M, G) + floor(M / 128)) ceil(N / 128) tiles of few rows an expert, (ceil(M / 256) + G) ceil(N / 256) of
# many.  Every second expert claims all rows: these are tiles enough for the experts below `last`, and for none from it on.
@pytest.mark.parametrize("M,G,N,K,last", [(1000, 32, 1280, 160, 10), (1000, 32, 96, 1024, 10), (2560, 8, 512, 160, 4)],
                         ids=["few_rows", "few_rows_split", "pairs"])
def test_no_more_tiles_than_the_launch_holds(M, G, N, K, last):
    """Ranges that overlap ask for several times the tiles that the launch and its counters were made for: those past the
    limit are left out.  The scales of the experts that come too late are NaN, which no row may show."""
    from mxfp8_microscaled_precision_gb300 import mxq
    off = torch.tensor([M * (g % 2) for g in range(G + 1)], device="cuda")
    bands, atoms = -(-M // 128) + G, -(-K // 128)
    a_q = torch.randint(0, 256, (M, 16 * -(-K // 32)), dtype=torch.uint8, device="cuda")
    a_s = torch.full((bands * atoms * 512,), 127, dtype=torch.uint8, device="cuda")
    b_q = torch.randint(0, 256, (G, N, 16 * -(-K // 32)), dtype=torch.uint8, device="cuda")
    b_s = torch.full((G, -(-N // 128) * atoms * 512), 127, dtype=torch.uint8, device="cuda")
    b_s[last:] = 255
    wide = torch.full((M + 64, N), 9.0, dtype=torch.bfloat16, device="cuda")
    mxq.grouped_gemm_mxfp4(a_q, a_s, b_q, b_s, off, N, K, out=wide[32:32 + M])
    assert not bool(wide.isnan().any())
    assert bool((wide[:32] == 9).all()) and bool((wide[32 + M:] == 9).all())
    # a call that keeps the rule, behind it: the first expert's product of all rows
    off = torch.tensor([0] + [M] * G, device="cuda")
    y = mxq.grouped_gemm_mxfp4(a_q, a_s, b_q, b_s, off, N, K)
    size = -(-M // 128) * atoms * 512
    assert torch.equal(y, mxq.gemm_mxfp4(a_q, a_s[:size], b_q[0], b_s[0], M, N, K))
    assert mxq.get_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("off", [[100, -2 ** 63, 100], [0, -2 ** 63, -2 ** 63 + 5], [2 ** 63 - 1, -2 ** 63, 2 ** 63 - 1], [99, -2 ** 63 + 1, 0]])
def test_ranges_that_end_before_they_start_have_no_columns(off, dtype):
    """However far before: the difference of such offsets may wrap around in 64 bits, and a range that seems long would be read
    behind the matrix."""
    from mxfp8_microscaled_precision_gb300 import mxq
    M, K, G = 100, 160, 2
    x = torch.randn(M, K, device="cuda").to(dtype)
    slots = -(-M // 128) + G
    q, s = torch.full((K, 64 * slots), 0x5A, dtype=torch.uint8, device="cuda"), torch.full((2 * slots * 512,), 0x5A, dtype=torch.uint8, device="cuda")
    mxq.quant_mxfp4_cols_grouped(x, torch.tensor(off, device="cuda"), out=(q, s))
    assert bool((q == 0x5A).all()) and bool((s == 0x5A).all())
    dw = mxq.grouped_gemm_mxfp4_wgrad(q, s, q, s, torch.tensor(off, device="cuda"), M)
    assert dw.shape == (G, K, K)
    assert mxq.get_device_status() == 0
