"""MXFP4 on the GPU: quantization and values bit by bit, products against 64 bits.

Tolerance of the products: the operands' products are exact, so with scales of a few powers of two every partial
sum of up to 4096 terms is a multiple of 2^-4 below 2^20 times that and FP32 holds it exactly, in any order: the result is the
exact sum rounded to BF16 once, and has to be equal.  With scales over a wide range the sum is off by at most
(K/32 + 64) 2^-22 of the sum of the terms' sizes (a rounding or truncation of the running sum for each instruction's
64 terms and for each joining of partial sums), plus 2^-8 of the result for BF16."""
import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest
import torch

import _fp4
from _util import gpu_or_skip

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gpu_or_skip()


def _matrix(R, C, dtype, seed, special=True):
    """Values of many sizes, and groups of the hard kinds."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, C, generator=g) * torch.exp2(torch.randint(-6, 7, (R, 1), generator=g).float())
    if special:
        flat = x.view(-1)
        at = torch.randperm(flat.numel(), generator=g)[:24].tolist()
        hard = [float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 6.0, -6.0, 3.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 2.0 ** -126,
                2.0 ** -130, -(2.0 ** -133), 3e38, -3.3e38, 6.0001, 1e-30, 2.0 ** 127, 1.5 * 2.0 ** 20]
        for i, v in zip(at, hard):
            flat[i] = v
        if R > 2:
            x[1] = 0.0
            x[2] = (torch.randint(-24, 25, (C,), generator=g).float() / 4)   # ties
        if R > 5:
            x[4] *= 2.0 ** -127
            x[5] *= 2.0 ** 120
    return x.to(dtype)


SHAPES = [(1, 1), (1, 32), (1, 33), (3, 31), (2, 64), (31, 5), (32, 32), (33, 97), (1, 4096), (8, 4096), (100, 130), (128, 128),
          (129, 127), (200, 321), (257, 1111), (130, 520), (64, 2085)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("R,C", SHAPES)
def test_quantization_along_both_axes(R, C, dtype):
    from mxfp8_microscaled_precision_gb300 import mxq
    x = _matrix(R, C, dtype, R * 7 + C)
    for layout in ("tiled", "rowmajor"):
        got = mxq.quant_mxfp4(x.cuda(), layout=layout)
        for (q, s), m in zip((got[:2], got[2:]), (x, x.t())):
            codes, scales = _fp4.quantize(_fp4.f64(m), "e2m1")
            assert np.array_equal(q.cpu().numpy(), _fp4.pack(codes))
            assert np.array_equal(s.cpu().numpy(), _fp4.tiled(scales) if layout == "tiled" else scales)
    row, col = mxq.quant_mxfp4(x.cuda(), col=False), mxq.quant_mxfp4(x.cuda(), row=False)
    assert row[2] is None and row[3] is None and col[0] is None and col[1] is None
    want = mxq.quant_mxfp4(x.cuda())
    for a, b in zip((*row[:2], *col[2:]), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("R,C", [(1, 40), (5, 4099), (8, 7168), (9, 300), (120, 256), (127, 4096), (129, 7000), (1216, 2048), (1217, 2048), (1000, 4097)])
def test_row_copies_of_few_rows(R, C, dtype):
    """Given outputs full of other values: the padding of tiled scales up to 128 rows and 4 groups is zero, whoever writes it."""
    from mxfp8_microscaled_precision_gb300 import mxq
    x = _matrix(R, C, dtype, R + C)
    codes, scales = _fp4.quantize(_fp4.f64(x), "e2m1")
    size = -(-R // 128) * -(-C // 128) * 512
    q, s = torch.full((R, 16 * -(-C // 32)), 0x5A, dtype=torch.uint8, device="cuda"), torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda")
    mxq.quant_mxfp4(x.cuda(), col=False, out=(q, s, None, None))
    assert np.array_equal(q.cpu().numpy(), _fp4.pack(codes))
    assert np.array_equal(s.cpu().numpy(), _fp4.tiled(scales))
    many = mxq.quant_mxfp4(x.cuda().expand(3, R, C), col=False)
    assert all(torch.equal(many[0][i], q) and torch.equal(many[1][i], s) for i in range(3))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("off,ld", [(0, 168), (1, 161), (2, 163), (8, 160), (3, 200), (5, 173)])
def test_rows_that_start_anywhere(off, ld, dtype):
    """Views into a wider buffer of NaN: what lies outside the rows is neither read into a group nor written."""
    from mxfp8_microscaled_precision_gb300 import mxq
    x = _matrix(70, 157, dtype, off)
    wide = torch.full((off + 70 * ld + 64,), float("nan"), dtype=dtype, device="cuda")
    view = wide[off:off + 70 * ld].view(70, ld)[:, :157]
    view.copy_(x)
    for a, b in zip(mxq.quant_mxfp4(view), mxq.quant_mxfp4(x.cuda())):
        assert torch.equal(a, b)


def test_batches_and_given_outputs():
    from mxfp8_microscaled_precision_gb300 import mxq
    x = torch.stack([_matrix(100, 77, torch.bfloat16, i) for i in range(5)]).cuda()
    each = [mxq.quant_mxfp4(m) for m in x]
    want = [torch.stack(p) for p in zip(*each)]
    for a, b in zip(mxq.quant_mxfp4(x), want):
        assert torch.equal(a, b)
    guard = [torch.full((t.numel() + 512,), 0xA5, dtype=torch.uint8, device="cuda") for t in want]
    out = tuple(g[256:256 + t.numel()].view(t.shape) for g, t in zip(guard, want))
    got = mxq.quant_mxfp4(x, out=out)
    for g, o, a, b in zip(guard, out, got, want):
        assert a is o and torch.equal(a, b) and bool((g[:256] == 0xA5).all()) and bool((g[-256:] == 0xA5).all())
    wide = torch.zeros(5, 100, 90, dtype=torch.bfloat16, device="cuda")[:, :, 3:80].copy_(x)
    for a, b in zip(mxq.quant_mxfp4(wide), want):
        assert torch.equal(a, b)
    assert [t.numel() for t in mxq.quant_mxfp4(x[:, :0])] == [0, 0, 0, 0]
    assert [t.numel() for t in mxq.quant_mxfp4(x[:0])] == [0, 0, 0, 0]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3", "e5m2"])
@pytest.mark.parametrize("R,C", [(1, 1), (3, 31), (5, 64), (130, 100), (7, 1111), (300, 256)])
def test_values(R, C, fmt, dtype):
    from mxfp8_microscaled_precision_gb300 import mxq
    rng = np.random.default_rng(R * 31 + C)
    G = -(-C // 32)
    four = fmt == "e2m1"
    codes = rng.integers(0, 16 if four else 256, (R, 32 * G)).astype(np.uint8)
    scales = rng.choice([0, 1, 2, 100, 120, 126, 127, 128, 140, 200, 230, 255], (R, G)).astype(np.uint8)
    want = _fp4.values(codes, scales, C, fmt)
    want = _fp4.bf16(want) if dtype == torch.bfloat16 else torch.from_numpy(want.astype(np.float32))
    width = 16 * G if four else C
    payload = torch.from_numpy(_fp4.pack(codes) if four else np.ascontiguousarray(codes[:, :C])).cuda()
    wide = torch.zeros(R, width + 36, dtype=torch.uint8, device="cuda")
    wide[:, 4:4 + width] = payload
    plain, tiles = torch.from_numpy(scales).cuda(), torch.from_numpy(_fp4.tiled(scales)).cuda()
    for q in (payload, wide[:, 4:4 + width]):
        for s, layout in ((plain, "rowmajor"), (tiles, "tiled"), (torch.cat([plain, plain], 1)[:, G:], "rowmajor")):
            got = mxq.dequant_1x32(q, s, C, fmt=fmt, layout=layout, dtype=dtype)
            assert got.dtype == dtype
            assert torch.equal(got.cpu().isnan(), want.isnan()) and torch.equal(got.cpu().nan_to_num(7.0, 5.0, -5.0), want.nan_to_num(7.0, 5.0, -5.0))
    out = torch.full((R, C + 3), 9.0, dtype=dtype, device="cuda")
    view = out[:, 1:1 + C]
    assert mxq.dequant_1x32(payload, tiles, C, fmt=fmt, dtype=dtype, out=view) is view
    assert torch.equal(view.cpu().nan_to_num(7.0, 5.0, -5.0), want.nan_to_num(7.0, 5.0, -5.0))
    assert bool((out[:, 0] == 9).all()) and bool((out[:, 1 + C:] == 9).all())


def test_values_restore_what_the_quantizers_made():
    from mxfp8_microscaled_precision_gb300 import mxq
    x = torch.randn(256, 320, device="cuda").bfloat16()
    q, s, _, _ = mxq.quant_1x32_dual(x, col=False)
    codes, scales = _fp4.quantize(_fp4.f64(x), "e4m3")
    assert np.array_equal(_fp4.f64(mxq.dequant_1x32(q, s, 320)), _fp4.values(codes, scales, 320, "e4m3"))
    q, s, _, _ = mxq.quant_1x32_dual_batched(x, col=False, fmt="e5m2", layout="rowmajor")
    codes, scales = _fp4.quantize(_fp4.f64(x), "e5m2")
    assert np.array_equal(_fp4.f64(mxq.dequant_1x32(q[0], s[0].view(256, 10), 320, fmt="e5m2", layout="rowmajor")),
                          _fp4.values(codes, scales, 320, "e5m2"))


# ---- products ---------------------------------------------------------------------------------------

def _operand(rng, R, K, **kw):
    codes, scales = _fp4.random_operand(rng, R, K, **kw)
    return (torch.from_numpy(_fp4.pack(codes)).cuda(), torch.from_numpy(_fp4.tiled(scales)).cuda(),
            torch.from_numpy(_fp4.values(codes, scales, K, "e2m1")))


PRODUCTS = [(1, 1, 1), (1, 8, 32), (1, 128, 64), (2, 16, 64), (3, 5, 33), (7, 130, 96), (8, 4096, 512), (16, 128, 128), (17, 127, 160),
            (31, 257, 2085), (33, 129, 257), (64, 256, 512), (65, 384, 300), (1, 7168, 1024), (100, 1003, 96), (127, 200, 4096), (128, 128, 4096),
            (129, 300, 1000), (200, 64, 2080), (255, 256, 256), (256, 256, 255), (257, 513, 300), (300, 260, 2085), (512, 768, 1024),
            (700, 1000, 777), (1024, 1024, 2048), (1500, 24, 320), (40, 5000, 608), (2049, 1537, 416)]


@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product_is_the_exact_sum_rounded_once(M, N, K):
    from mxfp8_microscaled_precision_gb300 import mxq
    rng = np.random.default_rng(M + 3 * N + 7 * K)
    a_q, a_s, a = _operand(rng, M, K)
    b_q, b_s, b = _operand(rng, N, K)
    want = _fp4.bf16((a.cuda() @ b.cuda().t()).cpu().numpy())
    got = mxq.gemm_mxfp4(a_q, a_s, b_q, b_s, M, N, K)
    assert torch.equal(got.cpu(), want)
    assert torch.equal(mxq.gemm_mxfp4(a_q, a_s, b_q, b_s, M, N, K), got)
    for pad, off in ((8, 0), (5, 1), (0, 3)):   # another row stride, another start
        wide = torch.full((off + M * (N + pad) + 8,), 9.0, dtype=torch.bfloat16, device="cuda")
        rows = wide[off:off + M * (N + pad)].view(M, N + pad)
        y = mxq.gemm_mxfp4(a_q, a_s, b_q, b_s, M, N, K, out=rows[:, :N])
        assert torch.equal(y, got)
        assert bool((rows[:, N:] == 9).all()) and bool((wide[:off] == 9).all()) and bool((wide[off + M * (N + pad):] == 9).all())
    assert mxq.get_device_status() == 0


@pytest.mark.parametrize("M,N,K", [(1, 512, 4096), (5, 300, 2085), (64, 1000, 1024), (300, 260, 1111), (1000, 700, 3000)])
def test_product_with_scales_of_every_size(M, N, K):
    from mxfp8_microscaled_precision_gb300 import mxq
    rng = np.random.default_rng(K)
    a_q, a_s, a = _operand(rng, M, K, lo=100, hi=150)
    b_q, b_s, b = _operand(rng, N, K, lo=90, hi=140)
    a, b = a.cuda(), b.cuda()
    ref, size = a @ b.t(), a.abs() @ b.abs().t()
    got = mxq.gemm_mxfp4(a_q, a_s, b_q, b_s, M, N, K).double()
    assert bool(((got - ref).abs() <= (K / 32 + 64) * 2.0 ** -22 * size + 2.0 ** -8 * ref.abs()).all())


@pytest.mark.parametrize("M,N,K", [(129, 8, 2048), (500, 520, 2113), (1024, 1024, 4128), (130, 4097, 4096), (1031, 129, 4500), (65, 1000, 4096),
                                   (257, 1500, 2050), (600, 31, 8192)])
def test_few_tiles_of_many_rows(M, N, K):
    """More rows than a tile has, K split over clusters: the exact sums (of up to 8192 terms: below 2^21 times their unit), into
    rows that leave in vectors and one by one."""
    from mxfp8_microscaled_precision_gb300 import mxq
    rng = np.random.default_rng(M * N)
    a_q, a_s, a = _operand(rng, M, K)
    b_q, b_s, b = _operand(rng, N, K)
    want = _fp4.bf16((a.cuda() @ b.cuda().t()).cpu().numpy())
    for ld in (N, N + 5):
        wide = torch.full((M + 1, ld), 7.0, dtype=torch.bfloat16, device="cuda")
        mxq.gemm_mxfp4(a_q, a_s, b_q, b_s, M, N, K, out=wide[:M, :N])
        assert torch.equal(wide[:M, :N].cpu(), want)
        assert (wide[M] == 7).all() and (wide[:, N:] == 7).all()


@pytest.mark.parametrize("M,N,K", [(2, 200, 160), (300, 300, 300)])
def test_a_nan_scale_makes_its_row_or_column_nan(M, N, K):
    from mxfp8_microscaled_precision_gb300 import mxq
    rng = np.random.default_rng(5)
    x = rng.standard_normal((M, K))
    w = rng.standard_normal((N, K))
    x[M - 1, K - 1], w[3, 2], w[N - 1, 0] = np.nan, np.inf, -np.inf
    xq, xs, _, _ = mxq.quant_mxfp4(torch.from_numpy(x).float().cuda(), col=False)
    wq, ws, _, _ = mxq.quant_mxfp4(torch.from_numpy(w).float().cuda(), col=False)
    nan = mxq.gemm_mxfp4(xq, xs, wq, ws, M, N, K).isnan().cpu()
    want = torch.zeros(M, N, dtype=torch.bool)
    want[M - 1], want[:, 3], want[:, N - 1] = True, True, True
    assert torch.equal(nan, want)


@pytest.mark.parametrize("M,N,K,ld", [(1024, 200, 320, 200), (1000, 456, 320, 456), (770, 232, 512, 240), (1024, 2024, 256, 2024)])
def test_ragged_widths_many_times(M, N, K, ld):
    """A last column tile that ends inside: chunks of the epilogue are left out, some rows leave in tiles and some by rows,
    and a buffer that was rewritten before its copy had read it would show now and then only."""
    from mxfp8_microscaled_precision_gb300 import mxq
    rng = np.random.default_rng(N)
    a_q, a_s, a = _operand(rng, M, K)
    b_q, b_s, b = _operand(rng, N, K)
    want = _fp4.bf16((a.cuda() @ b.cuda().t()).cpu().numpy()).cuda()
    y = torch.empty(M, ld, dtype=torch.bfloat16, device="cuda")[:, :N]
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(100):
        y.zero_()
        wrong += (mxq.gemm_mxfp4(a_q, a_s, b_q, b_s, M, N, K, out=y) != want).sum()
    assert int(wrong) == 0


@pytest.mark.parametrize("offset,pad", [(0, 0), (1, 0), (0, 1), (1, 1), (1, 2), (0, 3), (3, 8)])
@pytest.mark.parametrize("width", range(16))
def test_many_tiles_whose_rows_start_anywhere(width, offset, pad):
    """Every length of a row's last chunk of columns, on rows that start on a word and on rows that do not."""
    from mxfp8_microscaled_precision_gb300 import mxq
    M, N, K = 1291, 2033 + width, 96
    rng = np.random.default_rng(width)
    a_q, a_s, a = _operand(rng, M, K)
    b_q, b_s, b = _operand(rng, N, K)
    want = (a.cuda() @ b.cuda().t()).to(torch.bfloat16)   # sums of 96 terms: exact in 64 bits and in 32, rounded once
    ld = N + pad
    flat = torch.full((offset + M * ld + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = flat[offset:offset + M * ld].view(M, ld)
    mxq.gemm_mxfp4(a_q, a_s, b_q, b_s, M, N, K, out=y[:, :N])
    assert torch.equal(y[:, :N], want)
    assert bool((y[:, N:] == 7).all()) and bool((flat[:offset] == 7).all()) and bool((flat[offset + M * ld:] == 7).all())


@pytest.mark.parametrize("N,ld", [(4, 8), (13, 16), (2037, 2040), (250, 256), (1001, 1008)])
def test_experts_rows_wider_than_their_columns(N, ld):
    """Rows that start on 16 bytes with columns up to the middle of 16 bytes: what follows them stays."""
    from mxfp8_microscaled_precision_gb300 import mxq
    rng = np.random.default_rng(N)
    K, off = 96, torch.tensor([0, 500, 1100], device="cuda")
    x = torch.from_numpy(rng.integers(-12, 13, (1100, K)) / 2.0).bfloat16().cuda()
    b = [_operand(rng, N, K) for _ in range(2)]
    q, s = mxq.quant_mxfp4_grouped(x, off)
    v = mxq.dequant_1x32(*mxq.quant_mxfp4(x, col=False, layout="rowmajor")[:2], K, fmt="e2m1", layout="rowmajor").double()
    y = torch.full((1100, ld), 7.0, dtype=torch.bfloat16, device="cuda")
    mxq.grouped_gemm_mxfp4(q, s, torch.cat([e[0] for e in b]), torch.cat([e[1] for e in b]), off, N, K, out=y[:, :N])
    assert bool((y[:, N:] == 7).all())
    for g, (lo, hi) in enumerate(((0, 500), (500, 1100))):
        assert torch.equal(y[lo:hi, :N], (v[lo:hi] @ b[g][2].cuda().t()).to(torch.bfloat16))


def test_empty_products():
    from mxfp8_microscaled_precision_gb300 import mxq
    empty = torch.empty(0, dtype=torch.uint8, device="cuda")
    y = mxq.gemm_mxfp4(empty, empty, empty, empty, 5, 7, 0, out=torch.full((5, 9), 3.0, dtype=torch.bfloat16, device="cuda")[:, 1:8])
    assert bool((y == 0).all())
    q, s, _, _ = mxq.quant_mxfp4(torch.randn(5, 64, device="cuda"), col=False)
    assert mxq.gemm_mxfp4(empty, empty, q, s, 0, 5, 64).shape == (0, 5) and mxq.gemm_mxfp4(q, s, empty, empty, 5, 0, 64).shape == (5, 0)


def test_training_step_of_a_linear_layer():
    """The three products from one quantization of each matrix, against the values that the copies stand for."""
    from mxfp8_microscaled_precision_gb300 import mxq
    M, N, K = 333, 200, 450
    g = torch.Generator().manual_seed(1)
    x, w, dy = torch.randn(M, K, generator=g).cuda(), (0.05 * torch.randn(N, K, generator=g)).cuda(), torch.randn(M, N, generator=g).cuda()
    q = {n: mxq.quant_mxfp4(t.bfloat16()) for n, t in (("x", x), ("w", w), ("d", dy))}
    val = lambda n, c, cols: mxq.dequant_1x32(q[n][2 * c], q[n][2 * c + 1], cols, fmt="e2m1").double()  # noqa: E731
    for (a, ca), (b, cb), (m, n, k) in ((("x", 0), ("w", 0), (M, N, K)), (("d", 0), ("w", 1), (M, K, N)), (("d", 1), ("x", 1), (N, K, M))):
        got = mxq.gemm_mxfp4(*q[a][2 * ca:2 * ca + 2], *q[b][2 * cb:2 * cb + 2], m, n, k).double()
        va, vb = val(a, ca, k), val(b, cb, k)
        ref, size = va @ vb.t(), va.abs() @ vb.abs().t()
        assert bool(((got - ref).abs() <= (k / 32 + 64) * 2.0 ** -22 * size + 2.0 ** -8 * ref.abs()).all())


# ---- the experts' products ------------------------------------------------------------------------------

GROUPS = [([5], 0, 64, 96), ([0], 4, 40, 33), ([1, 1, 1], 0, 128, 64), ([0, 3, 0, 0, 70, 1, 0], 0, 130, 160), ([128, 128], 0, 256, 256),
          ([129, 127, 1], 3, 200, 300), ([300, 0, 40, 513], 7, 264, 520), ([0] * 30 + [2] + [0] * 30 + [90] + [0] * 5, 20, 136, 288),
          ([1, 0] * 100, 0, 128, 128), ([17] * 64, 0, 72, 96), ([0] * 1023 + [9], 1, 64, 64), ([1] * 1024, 0, 24, 32),
          ([2000, 5, 700], 100, 300, 777), ([3] * 8, 0, 1024, 2048), ([40, 1, 0, 64, 65, 31, 32, 33], 0, 513, 1000)]


@pytest.mark.parametrize("counts,behind,N,K", GROUPS, ids=lambda v: str(len(v)) + "x" + str(max(v)) if isinstance(v, list) else None)
def test_experts_products(counts, behind, N, K):
    from mxfp8_microscaled_precision_gb300 import mxq
    G, M = len(counts), sum(counts) + behind
    off = torch.tensor(np.cumsum([0] + counts), device="cuda")
    rng = np.random.default_rng(M + N)
    x = torch.from_numpy(rng.integers(-12, 13, (M, K)) / 2.0).bfloat16().cuda()   # halves up to 6, some of them rounded
    x[sum(counts):] = float("nan")
    a_q, a_s = mxq.quant_mxfp4_grouped(x, off, out=(torch.full((M, 16 * -(-K // 32)), 0x5A, dtype=torch.uint8, device="cuda"), None))
    each = [_operand(rng, N, K) for _ in range(G)] if G <= 200 else [_operand(rng, N, K)] * G
    b_q, b_s = torch.cat([e[0] for e in each]), torch.cat([e[1] for e in each])
    y = torch.full((M, N + 8), 9.0, dtype=torch.bfloat16, device="cuda")
    assert mxq.grouped_gemm_mxfp4(a_q, a_s, b_q, b_s, off, N, K, out=y[:, :N]).data_ptr() == y.data_ptr()
    plain_q, plain_s, _, _ = mxq.quant_mxfp4(x, col=False, layout="rowmajor")
    live = sum(counts)
    assert torch.equal(a_q[:live], plain_q[:live])
    assert bool((y[:, N:] == 9).all()) and bool((y[live:] == 9).all())
    v = mxq.dequant_1x32(plain_q, plain_s, K, fmt="e2m1", layout="rowmajor").double()
    for g in range(G):
        lo, hi = int(off[g]), int(off[g + 1])
        if hi > lo:
            want = _fp4.bf16((v[lo:hi] @ each[g][2].cuda().t()).cpu().numpy())
            assert torch.equal(y[lo:hi, :N].cpu(), want), g
            # the scales of the expert's rows in its own bands, beside the payload
            band = lo // 128 + g
            atoms = a_s.view(-1, -(-K // 128) * 512)[band:band + -(-(hi - lo) // 128)].reshape(-1)
            mine = _fp4.tiled(plain_s[lo:hi].cpu().numpy())
            used = _fp4.tiled(np.ones((hi - lo, plain_s.shape[1]), np.uint8)) > 0
            assert np.array_equal(atoms.cpu().numpy()[used], mine[used])
    odd = torch.full((M * (N + 3) + 1,), 9.0, dtype=torch.bfloat16, device="cuda")[1:].view(M, N + 3)
    assert torch.equal(mxq.grouped_gemm_mxfp4(a_q, a_s, b_q, b_s, off, N, K, out=odd[:, :N]), y[:, :N]) and bool((odd[:, N:] == 9).all())
    assert mxq.get_device_status() == 0


@pytest.mark.parametrize("K,ld,dtype", [(256, 256, torch.bfloat16), (300, 300, torch.bfloat16), (300, 317, torch.bfloat16), (520, 520, torch.float32),
                                        (45, 45, torch.float32)])
@pytest.mark.parametrize("counts,behind", [([3, 0, 70], 5), ([0, 0], 40), ([128], 1), ([64, 1], 200), ([500, 12], 0)])
def test_rows_of_no_expert_are_not_written(counts, behind, K, ld, dtype):
    """Payload rows behind the last expert and scales of rows that no expert has, whatever the rows hold."""
    from mxfp8_microscaled_precision_gb300 import mxq
    live, M, G = sum(counts), sum(counts) + behind, len(counts)
    x = torch.randn(M, ld, device="cuda").to(dtype)[:, :K]
    x[live:] = float("inf")
    off = torch.tensor(np.cumsum([0] + counts), device="cuda")
    bands, atoms = -(-M // 128) + G, -(-K // 128)
    q = torch.full((M, 16 * -(-K // 32)), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.full((bands * atoms * 512,), 0x5A, dtype=torch.uint8, device="cuda")
    mxq.quant_mxfp4_grouped(x, off, out=(q, s))
    assert bool((q[live:] == 0x5A).all())
    plain = mxq.quant_mxfp4(x, col=False, layout="rowmajor")
    assert torch.equal(q[:live], plain[0][:live])
    # byte of row r, group g of a band's atom: 16 (r % 32) + 4 (r / 32) + g
    r = torch.arange(128, device="cuda")
    at = (16 * (r % 32) + 4 * (r // 32))[:, None] + torch.arange(4, device="cuda")
    rows = s.view(bands, atoms, 512)[:, :, at]   # [band, atom, row, group]
    mine = torch.zeros(bands, 128, dtype=torch.bool, device="cuda")
    for g, n in enumerate(counts):
        first = int(off[g]) // 128 + g
        mine.view(-1)[128 * first:128 * first + n] = True
    assert bool((rows.permute(0, 2, 1, 3)[~mine] == 0x5A).all())


def test_no_rows_at_all():
    from mxfp8_microscaled_precision_gb300 import mxq
    off = torch.zeros(4, dtype=torch.int64, device="cuda")
    none = torch.empty(0, 96, dtype=torch.bfloat16, device="cuda")
    q, s = mxq.quant_mxfp4_cols_grouped(none, off)
    assert q.shape == (96, 3 * 64)
    y = torch.full((3, 96, 96), 9.0, dtype=torch.bfloat16, device="cuda")
    assert bool((mxq.grouped_gemm_mxfp4_wgrad(q.fill_(0x77), s.fill_(255), q, s, off, 0, out=y) == 0).all())
    q, s = mxq.quant_mxfp4_grouped(none, off)
    w, ws, _, _ = mxq.quant_mxfp4(torch.randn(3, 40, 96, device="cuda"), col=False)
    assert mxq.grouped_gemm_mxfp4(q, s, w, ws, off, 40, 96).shape == (0, 40)
    for shape in ((0, 64), (64, 0), (0, 0)):
        got = mxq.quant_mxfp4(torch.empty(shape, device="cuda"))
        assert got[0].shape == (shape[0], shape[1] // 2) and got[2].shape == (shape[1], shape[0] // 2)
        assert mxq.dequant_1x32(got[0], got[1], shape[1], fmt="e2m1").shape == shape
    assert mxq.get_device_status() == 0


CAPTURE = """
import sys, torch
from mxfp8_microscaled_precision_gb300 import mxq
x, w = torch.randn(200, 4096, device="cuda").bfloat16(), torch.randn(2, 300, 4096, device="cuda").bfloat16()
off = torch.tensor([0, 150, 200], device="cuda")
z, dy = torch.randn(50, 512, device="cuda").bfloat16(), torch.randn(50, 256, device="cuda").bfloat16()
side = torch.cuda.Stream()
def step():
    main = torch.cuda.current_stream()
    side.wait_stream(main)
    with torch.cuda.stream(side):                      # weights there, rows here
        k = mxq.quant_mxfp4(w)
        c = mxq.quant_mxfp4_cols_grouped(x[:, :300], off)
    q = mxq.quant_mxfp4(x.clone(), col=False)
    g = mxq.quant_mxfp4_grouped(x, off)
    main.wait_stream(side)
    few, many = mxq.gemm_mxfp4(q[0], q[1], k[0][0], k[1][0], 200, 300, 4096), mxq.gemm_mxfp4(k[2][0], k[3][0], k[2][1], k[3][1], 4096, 4096, 300)
    y = mxq.grouped_gemm_mxfp4(*g, k[0], k[1], off, 300, 4096)
    dw = mxq.grouped_gemm_mxfp4_wgrad(*c, *c, off, 200)
    a, zq, zs = mxq.activation(z)
    return (few, many, y, dw, a, *mxq.activation_backward(dy, zq, zs), mxq.dequant_1x32(k[0][0], k[1][0], 4096, fmt="e2m1"))
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):                          # no call was made before
    held = step()
for seed in range(3):
    for t in (x, w, z, dy):
        t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(seed)))
    for t in held:
        t.fill_(float("nan"))
    graph.replay()
    want = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, want)), [torch.equal(a, b) for a, b in zip(held, want)]
assert mxq.get_device_status() == 0
print("captured")
"""


def test_first_calls_inside_a_capture_that_forks():
    """In a process of its own: kernels' limits and the device's shape are looked up while the stream is captured, and
    launches follow copies and joins of streams there."""
    done = subprocess.run([sys.executable, "-c", CAPTURE], cwd=Path(__file__).resolve().parents[1], capture_output=True, text=True,
                          timeout=300)
    assert done.returncode == 0 and "captured" in done.stdout, done.stdout[-500:] + done.stderr[-2000:]


@pytest.mark.parametrize("counts,behind,M,N", [([5], 0, 64, 96), ([0], 4, 40, 33), ([1, 1, 1], 0, 128, 8), ([0, 3, 0, 0, 70, 1, 0], 0, 130, 160),
                                                ([128, 128], 0, 256, 256), ([129, 127, 1, 256], 3, 200, 300), ([300, 0, 40, 513], 7, 264, 520),
                                                ([1, 0] * 100, 0, 24, 40), ([33, 64, 65, 31, 32], 60, 513, 257), ([17] * 64, 0, 72, 1)],
                         ids=lambda v: str(len(v)) + "x" + str(max(v)) if isinstance(v, list) else None)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_experts_weight_gradients(counts, behind, M, N, dtype):
    """The column copies inside each expert bit by bit, and the products over its rows: of so few values and rows that FP32
    holds every partial sum."""
    from mxfp8_microscaled_precision_gb300 import mxq
    G, R = len(counts), sum(counts) + behind
    off = torch.tensor(np.cumsum([0] + counts), device="cuda")
    rng = np.random.default_rng(R + N)
    x, d = (torch.from_numpy(rng.integers(-12, 13, (R, n)) / 2.0).to(dtype).cuda() for n in (N, M))
    for t in (x, d):
        t[sum(counts):] = float("nan")
    bands = -(-R // 128) + G
    guard = torch.full((N * bands * 64 + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    a_q, a_s = mxq.quant_mxfp4_cols_grouped(d, off)
    b_q, b_s = mxq.quant_mxfp4_cols_grouped(x, off, out=(guard[256:-256].view(N, bands * 64), None))
    assert bool((guard[:256] == 0x5A).all()) and bool((guard[-256:] == 0x5A).all())
    y = mxq.grouped_gemm_mxfp4_wgrad(a_q, a_s, b_q, b_s, off, R)
    assert y.shape == (G, M, N)
    used = torch.full((N, bands * 64), False)
    for g in range(G):
        lo, hi = int(off[g]), int(off[g + 1])
        if hi == lo:
            assert bool((y[g] == 0).all())
            continue
        v = []
        for t in (d, x):
            codes, scales = _fp4.quantize(_fp4.f64(t[lo:hi].t()), "e2m1")
            v.append(_fp4.values(codes, scales, hi - lo, "e2m1"))
        slot, size = lo // 128 + g, -(-(hi - lo) // 128)
        want = np.zeros((N, 64 * size), np.uint8)
        want[:, :codes.shape[1] // 2] = _fp4.pack(codes)
        assert np.array_equal(b_q[:, 64 * slot:64 * (slot + size)].cpu().numpy(), want)
        used[:, 64 * slot:64 * (slot + size)] = True
        full = np.zeros((N, 4 * size), np.uint8)
        full[:, :scales.shape[1]] = scales
        atoms = b_s.view(-1, bands, 512)[:, slot:slot + size].reshape(-1).cpu().numpy()
        assert np.array_equal(atoms, _fp4.tiled(full))
        assert torch.equal(y[g].cpu(), _fp4.bf16(v[0] @ v[1].T)), g
    assert bool((b_q.cpu()[~used] == 0x5A).all())   # what is no expert's stays as it was
    assert mxq.get_device_status() == 0


def test_experts_input_gradients():
    """dX = dY W_g from the column copies of the stacked weights."""
    from mxfp8_microscaled_precision_gb300 import mxq
    G, R, N, K = 5, 300, 200, 330
    off = torch.tensor([0, 100, 100, 129, 299, 300], device="cuda")
    g = torch.Generator().manual_seed(2)
    w, dy = torch.randn(G, N, K, generator=g).cuda(), torch.randn(R, N, generator=g).cuda()
    _, _, w_q, w_s = mxq.quant_mxfp4(w, row=False)
    dx = mxq.grouped_gemm_mxfp4(*mxq.quant_mxfp4_grouped(dy, off), w_q, w_s, off, K, N)
    dq, ds, _, _ = mxq.quant_mxfp4(dy, col=False, layout="rowmajor")
    d = mxq.dequant_1x32(dq, ds, N, fmt="e2m1", layout="rowmajor").double()
    for e in range(G):
        lo, hi = int(off[e]), int(off[e + 1])
        v = mxq.dequant_1x32(w_q[e], w_s[e], N, fmt="e2m1").double()
        ref, size = d[lo:hi] @ v.t(), d[lo:hi].abs() @ v.abs().t()
        assert bool(((dx[lo:hi].double() - ref).abs() <= (N / 32 + 64) * 2.0 ** -22 * size + 2.0 ** -8 * ref.abs()).all())


@pytest.mark.parametrize("off", [[3, 50, 100], [0, 120, 60], [0, 50, 5000], [-10, 20, 100], [2 ** 62, -2 ** 62, 7], [100, 0, 0]])
def test_offsets_that_break_the_rule_stay_inside(off):
    """Rows are unspecified; what lies around the buffers stays as it was."""
    from mxfp8_microscaled_precision_gb300 import mxq
    M, N, K, G = 100, 96, 160, 2
    off = torch.tensor(off, device="cuda")
    x = torch.randn(M, K, device="cuda").bfloat16()
    sizes = [M * 80, (1 + G) * 2 * 512]
    guard = [torch.full((n + 2048,), 0xA5, dtype=torch.uint8, device="cuda") for n in sizes]
    q, s = guard[0][1024:-1024].view(M, 80), guard[1][1024:-1024]
    mxq.quant_mxfp4_grouped(x, off, out=(q, s))
    w = mxq.quant_mxfp4(torch.randn(G, N, K, device="cuda"), col=False)
    y = torch.full((M + 64, N), 9.0, dtype=torch.bfloat16, device="cuda")
    mxq.grouped_gemm_mxfp4(q, s, w[0], w[1], off, N, K, out=y[32:32 + M])
    sizes = [K * 64 * (1 + G), 2 * (1 + G) * 512]
    guard += [torch.full((n + 2048,), 0xA5, dtype=torch.uint8, device="cuda") for n in sizes]
    c, cs = guard[2][1024:-1024].view(K, -1), guard[3][1024:-1024]
    mxq.quant_mxfp4_cols_grouped(x, off, out=(c, cs))
    dw = torch.full((G + 2, K, K), 9.0, dtype=torch.bfloat16, device="cuda")
    mxq.grouped_gemm_mxfp4_wgrad(c, cs, c, cs, off, M, out=dw[1:1 + G])
    torch.cuda.synchronize()
    assert bool((y[:32] == 9).all()) and bool((y[32 + M:] == 9).all()) and bool((dw[0] == 9).all()) and bool((dw[-1] == 9).all())
    for g in guard:
        assert bool((g[:1024] == 0xA5).all()) and bool((g[-1024:] == 0xA5).all())
    assert mxq.get_device_status() == 0


# ---- streams, graphs, threads -----------------------------------------------------------------------------

def test_another_stream_and_a_captured_graph():
    from mxfp8_microscaled_precision_gb300 import mxq
    x, w = torch.randn(40, 500, device="cuda").bfloat16(), torch.randn(300, 500, device="cuda").bfloat16()
    off = torch.tensor([0, 11, 40], device="cuda")

    def step():
        q = mxq.quant_mxfp4(x, col=False)
        k = mxq.quant_mxfp4(w, col=False)
        g = mxq.quant_mxfp4_grouped(x, off)
        stacked = w.view(2, 150, 500)
        ws = mxq.quant_mxfp4(stacked, col=False)
        return (mxq.gemm_mxfp4(q[0], q[1], k[0], k[1], 40, 300, 500), mxq.grouped_gemm_mxfp4(*g, ws[0], ws[1], off, 150, 500),
                mxq.dequant_1x32(k[0], k[1], 500, fmt="e2m1"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = step()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(first, step()):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in range(3):
        x.copy_(torch.randn(40, 500, generator=torch.Generator().manual_seed(seed)))
        off.copy_(torch.tensor([0, 3 * seed, 40 - seed]))
        [h.fill_(5) for h in held]
        graph.replay()
        want = step()
        assert torch.equal(held[0], want[0]) and torch.equal(held[2], want[2])
        assert torch.equal(held[1][:40 - seed], want[1][:40 - seed]) and bool((held[1][40 - seed:] == 5).all())


def test_host_threads():
    import threading
    from mxfp8_microscaled_precision_gb300 import mxq
    jobs = []
    for M, N, K in ((1, 700, 1000), (300, 520, 600), (64, 256, 2048)):
        x, w = torch.randn(M, K, device="cuda"), torch.randn(N, K, device="cuda")
        k = mxq.quant_mxfp4(w, col=False)
        jobs.append((x, k, (M, N, K), mxq.gemm_mxfp4(*mxq.quant_mxfp4(x, col=False)[:2], *k[:2], M, N, K)))
    torch.cuda.synchronize()
    bad = []

    def work(x, k, size, want):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(300):
                got = mxq.gemm_mxfp4(*mxq.quant_mxfp4(x, col=False)[:2], *k[:2], *size)
            torch.cuda.current_stream().synchronize()
            if not torch.equal(got, want):
                bad.append(size)
    threads = [threading.Thread(target=work, args=j) for j in jobs]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert bad == []


@pytest.mark.parametrize("call", ["payload", "scales", "experts", "given", "batch"])
def test_refusals(call):
    from mxfp8_microscaled_precision_gb300 import mxq
    x = torch.randn(64, 96, device="cuda")
    q, s, _, _ = mxq.quant_mxfp4(x, col=False)
    off = torch.tensor([0, 64], device="cuda")
    calls = {"payload": lambda: mxq.gemm_mxfp4(q[:63], s, q, s, 64, 64, 96), "scales": lambda: mxq.gemm_mxfp4(q, s[:-1], q, s, 64, 64, 96),
             "experts": lambda: mxq.grouped_gemm_mxfp4(q, s, q, s, torch.zeros(2000, dtype=torch.int64, device="cuda"), 64, 96),
             "given": lambda: mxq.gemm_mxfp4(q, s, q, s, 64, 64, 96, out=torch.empty(64, 64, device="cuda")),
             "batch": lambda: mxq.quant_mxfp4(x, col=False, out=(None, None, q, s))}
    with pytest.raises(ValueError):
        calls[call]()
    with pytest.raises(ValueError):
        mxq.quant_mxfp4_grouped(x, off.int())
    with pytest.raises(ValueError):
        mxq.quant_mxfp4(x.t())
