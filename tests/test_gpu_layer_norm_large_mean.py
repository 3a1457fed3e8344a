"""Layer norm's gradients where the mean is far above the spread, against numpy in 64 bits.

The gradients take mean and rstd as inputs: h = (x - mean) rstd, a difference and a product that round once
each, so h is off by 3 u |h| at most (u = 2^-24, the second order included), however large the mean is.
Beside that, with n = cols / 1024 + 64 the longest chain of rounded additions in a row's sum:
  dx   4 u (|u| + |m1| + |h m2|) + n u mean|u| + |h| (n u mean|u h| + mean(|u| eh)) + eh |m2|, times rstd;
  dw   (rows / 304 + 320) u sum|dy h| + sum(|dy| eh),  db  (rows / 304 + 320) u sum|dy|.
A form that rounds mean * rstd (x rstd - mean rstd) is off by u |mean| rstd / 2: 1e-4 here, where 3 u |h| is 2e-7."""
import numpy as np
import pytest
import torch

from _util import gpu_or_skip

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16 = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gpu_or_skip()


def _f64(t):
    return t.double().cpu().numpy()


# widths of every backward kernel: parts of a warp, the ring with a row kept in registers (on and off the
# 16-byte grid, groups of several sizes) and read twice, the longest rows
@pytest.mark.parametrize("C", [8, 64, 97, 500, 513, 1024, 1111, 4096, 4100, 5120, 8192, 8999, 12288, 16384, 20001])
@pytest.mark.parametrize("M", [2, 330])
@pytest.mark.parametrize("dtype,wdtype", [(torch.float32, torch.float32), (torch.float32, torch.bfloat16),
                                          (torch.bfloat16, torch.float32)])
def test_large_mean(M, C, dtype, wdtype):
    from mxfp8_microscaled_precision_gb300 import mxq
    g = torch.Generator().manual_seed(M + C)
    # BF16 has 8 bits: around 4096 its values are 32 apart
    spread = 1.0 if dtype == torch.float32 else 64.0
    x = (4096.0 + spread * torch.randn(M, C, generator=g)).to(dtype).cuda()
    w = (1 + 0.3 * torch.randn(C, generator=g)).to(wdtype).cuda()
    dy = torch.randn(M, C, generator=g).to(dtype).cuda()
    # the statistics in 64 bits, rounded once: what they are off by is not the backward pass's
    X = _f64(x)
    mean = torch.from_numpy(X.mean(1)).float().cuda()
    rstd = torch.from_numpy(1 / np.sqrt(((X - X.mean(1, keepdims=True)) ** 2).mean(1) + 1e-5)).float().cuda()
    dx, dw, db = (_f64(t) for t in mxq.layer_norm_backward(dy, x, w, mean, rstd))
    D, W, m, r = _f64(dy), _f64(w), _f64(mean)[:, None], _f64(rstd)[:, None]
    n = C / 1024 + 64
    h = (X - m) * r
    eh = 3 * U * np.abs(h)
    u = D * W
    m1, m2 = u.mean(1, keepdims=True), (u * h).mean(1, keepdims=True)
    e1 = n * U * np.abs(u).mean(1, keepdims=True)
    e2 = n * U * np.abs(u * h).mean(1, keepdims=True) + (np.abs(u) * eh).mean(1, keepdims=True)
    ref = r * (u - m1 - h * m2)
    bound = r * (4 * U * (np.abs(u) + np.abs(m1) + np.abs(h * m2)) + e1 + np.abs(h) * e2 + eh * np.abs(m2))
    if dtype == torch.bfloat16:
        bound = bound + BF16 * np.abs(ref)
    s = (M / 304 + 320) * U
    assert np.all(np.abs(dw - (D * h).sum(0)) <= s * np.abs(D * h).sum(0) + (np.abs(D) * eh).sum(0) + 1e-37)
    assert np.all(np.abs(db - D.sum(0)) <= s * np.abs(D).sum(0) + 1e-37)
    assert np.all(np.abs(dx - ref) <= bound + 1e-37)
