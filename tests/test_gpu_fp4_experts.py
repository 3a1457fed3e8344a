"""The experts' products in MXFP4 where the choice of the kernel changes and in the input gradient's form.

Equalities: codes up to 6, all scales 1, so every sum of up to 4096 products is a multiple of 1/4 below 2^18 and FP32 holds
it in any order.  Else a sum is off by at most (N/32 + 64) 2^-22 of the sum of the terms' sizes (a rounding or truncation
of the running sum for each instruction's 64 terms and for each joining of partial sums), plus 2^-8 of the result for BF16."""
import numpy as np
import pytest
import torch

from _util import gpu_or_skip

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gpu_or_skip()


@pytest.mark.parametrize("N,K", [(1024, 4096), (4096, 512), (200, 1111)])
@pytest.mark.parametrize("M", [1, 47, 48, 49, 64, 65, 129, 257])
def test_one_expert_is_the_dense_product(M, N, K):
    """48 rows an expert and fewer take one kernel, more the other; the dense product has its own rule."""
    from mxfp8_microscaled_precision_gb300 import mxq
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    width, atoms = 16 * -(-K // 32), -(-K // 128) * 512

    def operand(rows, bands):
        q = torch.randint(0, 256, (rows, width), dtype=torch.uint8, device="cuda", generator=gen)
        q[:, K // 2:] = 0   # past K; of an odd K the last element's byte holds one code
        if K % 2:
            q[:, K // 2] = torch.randint(0, 16, (rows,), dtype=torch.uint8, device="cuda", generator=gen)
        return q, torch.full((bands * atoms,), 127, dtype=torch.uint8, device="cuda")

    (a, sa), (b, sb) = operand(M, -(-M // 128) + 1), operand(N, -(-N // 128))
    dense = mxq.gemm_mxfp4(a, sa[:-(-M // 128) * atoms], b, sb, M, N, K)
    off = torch.tensor([0, M], device="cuda")
    assert torch.equal(mxq.grouped_gemm_mxfp4(a, sa, b, sb, off, N, K), dense)
    code = torch.stack((a & 15, a >> 4), -1).view(M, -1), torch.stack((b & 15, b >> 4), -1).view(N, -1)
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    va, vb = (table[(c & 7).long()] * (1.0 - 2.0 * (c >> 3).double()) for c in code)
    assert torch.equal(dense, (va @ vb.t()).to(torch.bfloat16))


@pytest.mark.parametrize("N,K", [(768, 4096), (300, 2085), (1024, 4064), (130, 4000)])
@pytest.mark.parametrize("counts,behind", [([200], 0), ([130, 0, 1], 7), ([1, 255], 0), ([500], 30), ([0, 129, 128, 127], 0), ([300, 300], 100)])
def test_few_experts_of_many_rows_and_long_rows(counts, behind, N, K):
    """Few tiles, each with K split over a cluster, of experts that start and end inside a tile; rows of no expert stay."""
    from mxfp8_microscaled_precision_gb300 import mxq
    G, live = len(counts), sum(counts)
    M = live + behind
    gen = torch.Generator(device="cuda").manual_seed(M + K)
    off = torch.tensor(np.cumsum([0] + counts), device="cuda")
    # halves up to 6, with a 6 in each group of 32: scales of 1, values as they are
    x, w = (torch.randint(-8, 9, (n, K), generator=gen, device="cuda").double() / 2 for n in (M, G * N))
    x[:, ::32], w[:, ::32] = 6, 6
    for t in (x, w):
        t[t.abs() == 3.5] = 4.0
        t[t.abs() == 2.5] = 2.0
    y = torch.full((M, N + 8), 9.0, dtype=torch.bfloat16, device="cuda")
    x[live:] = float("inf")
    q = mxq.quant_mxfp4_grouped(x.bfloat16(), off)
    wq, ws, _, _ = mxq.quant_mxfp4(w.bfloat16().view(G, N, K), col=False)
    mxq.grouped_gemm_mxfp4(*q, wq, ws, off, N, K, out=y[:, :N])
    assert bool((y[live:] == 9).all()) and bool((y[:, N:] == 9).all())
    for g, n in enumerate(counts):
        lo = int(off[g])
        assert torch.equal(y[lo:lo + n, :N], (x[lo:lo + n] @ w[g * N:(g + 1) * N].t()).to(torch.bfloat16))
    assert mxq.get_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("counts,behind,N,K", [([1, 0, 2], 1, 64, 96), ([48, 48, 0], 0, 130, 515), ([100, 49, 3], 5, 257, 320),
                                               ([0, 0, 300], 40, 1000, 77), ([700, 1, 0], 0, 520, 1024)])
def test_input_gradients(counts, behind, N, K, dtype):
    """dX = dY W_g with the column copies of stacked weights; rows of no expert stay as they are."""
    from mxfp8_microscaled_precision_gb300 import mxq
    G, R = len(counts), sum(counts) + behind
    gen = torch.Generator().manual_seed(N)
    off = torch.tensor(np.cumsum([0] + counts), device="cuda")
    w = (0.05 * torch.randn(G, N, K, generator=gen)).to(dtype).cuda()
    dy = torch.randn(R, N, generator=gen).to(dtype).cuda()
    dy[sum(counts):] = float("nan")
    _, _, w_q, w_s = mxq.quant_mxfp4(w, row=False)
    dx = torch.full((R, K + 3), 9.0, dtype=torch.bfloat16, device="cuda")
    mxq.grouped_gemm_mxfp4(*mxq.quant_mxfp4_grouped(dy, off), w_q, w_s, off, K, N, out=dx[:, :K])
    assert bool((dx[sum(counts):] == 9).all()) and bool((dx[:, K:] == 9).all())
    q, s, _, _ = mxq.quant_mxfp4(dy, col=False, layout="rowmajor")
    d = mxq.dequant_1x32(q, s, N, fmt="e2m1", layout="rowmajor").double()
    for g, n in enumerate(counts):
        if n:
            lo = int(off[g])
            v = mxq.dequant_1x32(w_q[g], w_s[g], N, fmt="e2m1").double()
            ref, size = d[lo:lo + n] @ v.t(), d[lo:lo + n].abs() @ v.abs().t()
            assert bool(((dx[lo:lo + n, :K].double() - ref).abs() <= (N / 32 + 64) * 2.0 ** -22 * size + 2.0 ** -8 * ref.abs()).all())
    assert mxq.get_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("counts,K", [([3, 0, 70, 128], 96), ([129, 300, 1], 515), ([0, 40], 1000)])
def test_values_of_one_experts_rows(counts, K, dtype):
    """A payload with scales by expert, read back an expert at a time: its rows, and the scales from its first band on."""
    from mxfp8_microscaled_precision_gb300 import mxq
    off = torch.tensor(np.cumsum([0] + counts), device="cuda")
    x = torch.randn(sum(counts), K, device="cuda").to(dtype)
    q, s = mxq.quant_mxfp4_grouped(x, off)
    atoms = -(-K // 128) * 512
    for g, n in enumerate(counts):
        lo = int(off[g])
        first = lo // 128 + g
        want = mxq.quant_mxfp4(x[lo:lo + n], col=False, layout="rowmajor")[:2]
        got = mxq.dequant_1x32(q[lo:lo + n], s[first * atoms:(first + -(-n // 128)) * atoms], K, fmt="e2m1", dtype=torch.float32)
        assert torch.equal(got, mxq.dequant_1x32(*want, K, fmt="e2m1", layout="rowmajor", dtype=torch.float32))
