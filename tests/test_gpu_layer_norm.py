"""Layer norm and its gradients on the GPU (mxq.layer_norm, layer_norm_backward)
against numpy in 64 bits.

Tolerances, with u = 2^-24 and n = cols / 1024 + 64 (the longest chain of rounded additions
in a row's sum: a thread's share and the trees over the block):
  mean  n u mean|x| =: dm;  rstd  (n + 8) u + dm rstd relative (dm enters the
  centred squares once, to first order 2 dm mean|x - mean| / var <= 2 dm rstd; halved by the root);
  y     |weight| rstd (dm + 2 u (|x| + |mean|)) + (n + 16 + dm rstd / u) u |h weight| + 2 u |shift|;
  the gradients take mean and rstd as inputs, so h is off by eh = 2 u (|x| + |mean|) rstd + 2 u |h|,
  the row means by n u mean|.| and mean(|u| eh), the column sums by (rows / 304 + 320) u sum|.|.
BF16 results add half a unit in the last place, 2^-8 relative."""
import numpy as np
import pytest
import torch

from _util import gpu_or_skip

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16 = 2.0 ** -8

SHAPES = [(1, 1), (1, 8), (3, 7), (2, 32), (1, 4096), (9, 255), (5, 513), (33, 1024), (4, 1111), (7, 4096), (130, 4104),
          (305, 257), (700, 2048), (1000, 64), (3, 7168), (2, 8193), (2, 16384), (3, 20001), (2, 32768), (2, 32769),
          (310, 40000)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gpu_or_skip()


def _f64(t):
    return t.double().cpu().numpy()


def _problem(M, C, dtype, wdtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(M, C, generator=g) * (0.2 + 4 * torch.rand(M, 1, generator=g)) + 3 * torch.randn(M, 1, generator=g))
    w = 1 + 0.3 * torch.randn(C, generator=g)
    b = 0.5 * torch.randn(C, generator=g)
    dy = torch.randn(M, C, generator=g)
    return x.to(dtype).cuda(), w.to(wdtype).cuda(), b.to(wdtype).cuda(), dy.to(dtype).cuda()


def _check_forward(x, w, b, eps, y, mean, rstd):
    X = _f64(x)
    C = X.shape[1]
    W = _f64(w) if w is not None else np.ones(C)
    B = _f64(b) if b is not None else np.zeros(C)
    n = C / 1024 + 64
    m = X.mean(1, keepdims=True)
    r = 1 / np.sqrt(((X - m) ** 2).mean(1, keepdims=True) + eps)
    dm = n * U * np.abs(X).mean(1, keepdims=True)
    assert np.all(np.abs(_f64(mean) - m[:, 0]) <= dm[:, 0])
    assert np.all(np.abs(_f64(rstd) / r[:, 0] - 1) <= ((n + 8) * U + dm * r)[:, 0])
    h = (X - m) * r
    ref = h * W + B
    bound = (np.abs(W) * r * (dm + 2 * U * (np.abs(X) + np.abs(m))) + ((n + 16) * U + dm * r) * np.abs(h * W)
             + 2 * U * np.abs(B))
    if y.dtype == torch.bfloat16:
        bound = bound + BF16 * np.abs(ref)
    assert np.all(np.abs(_f64(y) - ref) <= bound + 1e-37), np.abs(_f64(y) - ref).max()


def _check_backward(dy, x, w, mean, rstd, dx, dw, db):
    X, D, m, r = _f64(x), _f64(dy), _f64(mean)[:, None], _f64(rstd)[:, None]
    M, C = X.shape
    W = _f64(w) if w is not None else np.ones(C)
    n = C / 1024 + 64
    h = (X - m) * r
    eh = 2 * U * (np.abs(X) + np.abs(m)) * r + 2 * U * np.abs(h)
    u = D * W
    m1, m2 = u.mean(1, keepdims=True), (u * h).mean(1, keepdims=True)
    e1 = n * U * np.abs(u).mean(1, keepdims=True)
    e2 = n * U * np.abs(u * h).mean(1, keepdims=True) + (np.abs(u) * eh).mean(1, keepdims=True)
    ref = r * (u - m1 - h * m2)
    bound = r * (4 * U * (np.abs(u) + np.abs(m1) + np.abs(h * m2)) + e1 + np.abs(h) * e2 + eh * np.abs(m2))
    if dx.dtype == torch.bfloat16:
        bound = bound + BF16 * np.abs(ref)
    assert np.all(np.abs(_f64(dx) - ref) <= bound + 1e-37), np.abs(_f64(dx) - ref).max()
    s = (M / 304 + 320) * U
    assert np.all(np.abs(_f64(dw) - (D * h).sum(0)) <= s * np.abs(D * h).sum(0) + (np.abs(D) * eh).sum(0) + 1e-37)
    assert np.all(np.abs(_f64(db) - D.sum(0)) <= s * np.abs(D).sum(0) + 1e-37)


@pytest.mark.parametrize("dtype,wdtype", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                          (torch.float32, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("M,C", SHAPES)
def test_layer_norm_and_gradients(M, C, dtype, wdtype):
    from mxfp8_microscaled_precision_gb300 import mxq
    x, w, b, dy = _problem(M, C, dtype, wdtype, M + C)
    y, mean, rstd = mxq.layer_norm(x, w, b, eps=1e-5)
    assert y.dtype == dtype
    _check_forward(x, w, b, 1e-5, y, mean, rstd)
    dx, dw, db = mxq.layer_norm_backward(dy, x, w, mean, rstd)
    _check_backward(dy, x, w, mean, rstd, dx, dw, db)


@pytest.mark.parametrize("dtype,wdtype", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                          (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("M,C", [(4000, 520), (3000, 640), (2001, 2048), (1300, 7168), (1111, 1111), (2500, 515),
                                 (1531, 4097), (900, 8999), (700, 16384), (9000, 130), (6001, 257), (500, 12345)])
def test_many_rows(M, C, dtype, wdtype):
    """Every block walks over many rows: more than the shared memory holds at a time."""
    from mxfp8_microscaled_precision_gb300 import mxq
    x, w, b, dy = _problem(M, C, dtype, wdtype, M + C)
    y, mean, rstd = mxq.layer_norm(x, w, b, eps=1e-5)
    _check_forward(x, w, b, 1e-5, y, mean, rstd)
    one = mxq.layer_norm_backward(dy, x, w, mean, rstd)
    _check_backward(dy, x, w, mean, rstd, *one)
    assert all(torch.equal(p, q) for p, q in zip(one, mxq.layer_norm_backward(dy, x, w, mean, rstd)))
    assert mxq.get_device_status() == 0


@pytest.mark.parametrize("M,C,dtype,wdtype", [
    (700, 5120, torch.bfloat16, torch.bfloat16), (613, 4999, torch.bfloat16, torch.float32),
    (500, 4616, torch.float32, torch.float32), (457, 5121, torch.bfloat16, torch.bfloat16),
    (3000, 40, torch.bfloat16, torch.float32), (2999, 33, torch.bfloat16, torch.float32), (5000, 9, torch.float32, torch.bfloat16),
    (306, 24000, torch.bfloat16, torch.float32), (310, 25999, torch.bfloat16, torch.float32)])
def test_rows_of_every_grouping(M, C, dtype, wdtype):
    """Two groups of 320 threads; parameters kept in shared memory for parts of a warp, for a whole block, and
    too long for it."""
    test_many_rows(M, C, dtype, wdtype)


def test_without_weight_or_shift():
    from mxfp8_microscaled_precision_gb300 import mxq
    for C in (96, 97):
        x, w, b, dy = _problem(11, C, torch.bfloat16, torch.float32, C)
        for ww, bb in ((None, None), (w, None), (None, b)):
            y, mean, rstd = mxq.layer_norm(x, ww, bb, eps=1e-3)
            _check_forward(x, ww, bb, 1e-3, y, mean, rstd)
            _check_backward(dy, x, ww, mean, rstd, *mxq.layer_norm_backward(dy, x, ww, mean, rstd))


def test_gradients_against_differences():
    """Central differences in 64 bits of sum(dy * y): step h, an error of h^2 times third
    derivatives (below 100 here) and 1e-15 / h; the kernel's FP32 adds below 1e-5."""
    from mxfp8_microscaled_precision_gb300 import mxq
    M, C, h, eps = 3, 24, 1e-5, 1e-5
    x, w, b, dy = _problem(M, C, torch.float32, torch.float32, 8)
    _, mean, rstd = mxq.layer_norm(x, w, b, eps)
    dx, dw, db = (_f64(t) for t in mxq.layer_norm_backward(dy, x, w, mean, rstd))
    X, W, B, D = _f64(x), _f64(w), _f64(b), _f64(dy)

    def loss(X, W, B):
        m = X.mean(1, keepdims=True)
        return (D * ((X - m) / np.sqrt(((X - m) ** 2).mean(1, keepdims=True) + eps) * W + B)).sum()

    def slope(which, at):
        out = []
        for sgn in (1, -1):
            a = [X.copy(), W.copy(), B.copy()]
            a[which][at] += sgn * h
            out.append(loss(*a))
        return (out[0] - out[1]) / (2 * h)

    for i in range(C):
        for t in range(M):
            assert abs(slope(0, (t, i)) - dx[t, i]) <= 2e-5 * max(1.0, np.abs(dx).max())
        assert abs(slope(1, i) - dw[i]) <= 2e-5 * max(1.0, np.abs(dw).max())
        assert abs(slope(2, i) - db[i]) <= 2e-5 * max(1.0, np.abs(db).max())


def test_constant_rows_and_a_large_mean():
    """No variance: rstd = 1 / sqrt(eps), y = shift.  A mean far above the spread does not
    cancel: the centred squares are summed."""
    from mxfp8_microscaled_precision_gb300 import mxq
    for C in (64, 77, 33000):
        x = torch.full((3, C), 5.0, device="cuda")
        b = torch.randn(C, device="cuda")
        y, mean, rstd = mxq.layer_norm(x, torch.ones_like(b), b, eps=1e-4)
        assert torch.equal(mean, torch.full_like(mean, 5.0)) and torch.equal(y, b.expand(3, C))
        assert torch.all((rstd - 100).abs() < 1e-3)
        g = torch.randn(4, C, generator=torch.Generator().manual_seed(C)).cuda()
        big = 4096.0 + g
        y, mean, rstd = mxq.layer_norm(big)
        _check_forward(big, None, None, 1e-5, y, mean, rstd)


def test_nan_and_inf_stay_in_their_rows():
    from mxfp8_microscaled_precision_gb300 import mxq
    for C in (128, 129):
        x, w, b, dy = _problem(6, C, torch.bfloat16, torch.bfloat16, C)
        clean = mxq.layer_norm(x, w, b)[0]
        x[1, 3], x[4, 100] = float("nan"), float("inf")
        y, mean, rstd = mxq.layer_norm(x, w, b)
        keep = [0, 2, 3, 5]
        assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[1]).all() and torch.isnan(y[4]).all()
        dx, _, db = mxq.layer_norm_backward(dy, x, w, mean, rstd)
        assert torch.isfinite(dx[keep]).all() and torch.isfinite(db).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("C,pad,shift", [(64, 8, 0), (64, 3, 0), (64, 8, 1), (1024, 16, 8), (65, 8, 0), (4097, 2, 3),
                                         (32780, 4, 1)])
def test_strides_alignment_and_in_place(C, pad, shift, dtype):
    from mxfp8_microscaled_precision_gb300 import mxq
    M = 9
    x, w, b, dy = _problem(M, C, dtype, torch.float32, C + pad)

    def wide(t, fill):
        big = torch.full((M, C + pad + shift), fill, dtype=dtype, device="cuda")
        big[:, shift:shift + C] = t
        return big, big[:, shift:shift + C]

    _, vx = wide(x, float("nan"))
    _, vd = wide(dy, float("nan"))
    big, vy = wide(torch.zeros_like(x), 7.0)
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    mxq.layer_norm(vx, w, b, out=(vy, mean, rstd))
    _check_forward(x, w, b, 1e-5, vy, mean, rstd)
    assert (big[:, :shift] == 7).all() and (big[:, shift + C:] == 7).all()
    big, vg = wide(torch.zeros_like(x), 7.0)
    _check_backward(dy, x, w, mean, rstd, *mxq.layer_norm_backward(vd, vx, w, mean, rstd, out=vg))
    assert (big[:, :shift] == 7).all() and (big[:, shift + C:] == 7).all()
    # in place: the same answers
    y, dx = mxq.layer_norm(vx, w, b)[0], mxq.layer_norm_backward(vd, vx, w, mean, rstd)
    again = mxq.layer_norm_backward(vd, vx, w, mean, rstd, out=vd)
    assert all(torch.equal(p, q) for p, q in zip(again, dx))
    assert torch.equal(mxq.layer_norm(vx, w, b, out=(vx, None, None))[0], y)


def test_parameters_at_any_element():
    from mxfp8_microscaled_precision_gb300 import mxq
    x, w, b, dy = _problem(5, 512, torch.bfloat16, torch.bfloat16, 3)
    flat = torch.zeros(1100, dtype=torch.bfloat16, device="cuda")
    w1, b1 = flat[1:513], flat[515:1027]
    w1.copy_(w), b1.copy_(b)
    one, two = mxq.layer_norm(x, w, b), mxq.layer_norm(x, w1, b1)
    assert all(torch.equal(p, q) for p, q in zip(one, two))
    one, two = (mxq.layer_norm_backward(dy, x, v, *one[1:]) for v in (w, w1))
    assert all(torch.equal(p, q) for p, q in zip(one, two))


def test_empty_same_answer_twice_and_refusals():
    from mxfp8_microscaled_precision_gb300 import mxq
    w = torch.ones(32, device="cuda")
    e = torch.empty(0, 32, device="cuda")
    y, mean, rstd = mxq.layer_norm(e, w, w)
    assert y.shape == (0, 32)
    dx, dw, db = mxq.layer_norm_backward(e, e, w, mean, rstd)
    assert dx.shape == (0, 32) and (dw == 0).all() and (db == 0).all()
    x, w, b, dy = _problem(5000, 96, torch.bfloat16, torch.float32, 1)
    y, mean, rstd = mxq.layer_norm(x, w, b)
    one, two = (mxq.layer_norm_backward(dy, x, w, mean, rstd) for _ in range(2))
    assert all(torch.equal(p, q) for p, q in zip(one, two))
    for call in (lambda: mxq.layer_norm(x.half()), lambda: mxq.layer_norm(x[0]), lambda: mxq.layer_norm(x.t()),
                 lambda: mxq.layer_norm(x, w[:95]), lambda: mxq.layer_norm(x, w, b.bfloat16()),
                 lambda: mxq.layer_norm(x, eps=-1.0), lambda: mxq.layer_norm(x, eps=float("nan")),
                 lambda: mxq.layer_norm(x.cpu()), lambda: mxq.layer_norm(x, w.double(), b.double()),
                 lambda: mxq.layer_norm_backward(dy.float(), x, w, mean, rstd),
                 lambda: mxq.layer_norm_backward(dy[:10], x, w, mean, rstd),
                 lambda: mxq.layer_norm_backward(dy, x, w, mean[:10], rstd),
                 lambda: mxq.layer_norm_backward(dy, x, w, mean.double(), rstd)):
        with pytest.raises(ValueError):
            call()
