"""Rows into expert order and back on the GPU (mxq.moe_plan, moe_dispatch,
moe_combine, moe_combine_backward) against numpy in 64 bits.

The plan and dispatch move values and are exact.  combine is a sum of k products
in FP32: |error| <= (k + 1) 2^-24 sum |w y|, a dot product over H elements in a tree
of at most H / 32 + 5 additions: (H / 32 + 40) 2^-24 sum |a b|; BF16 results add half a
unit in the last place, 2^-8 relative (2^-9 would do)."""
import numpy as np
import pytest
import torch

from _util import gpu_or_skip

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
BF16 = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    gpu_or_skip()


def _ids(T, k, E, seed, dropped=0.0, wide=None):
    """k different experts per token, of the first `wide` only where given; -1 in some tokens."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.rand(T, wide or E, generator=g).argsort(1)[:, :k].to(torch.int32)
    ids[torch.rand(T, generator=g) < dropped] = -1
    if dropped:   # and in single places
        ids[torch.rand(T, k, generator=g) < dropped / 2] = -1
    return ids.cuda()


def _plan64(ids, E):
    flat = ids.cpu().numpy().reshape(-1)
    key = np.where((flat < 0) | (flat >= E), E, flat)
    order = np.argsort(key, kind="stable")
    row = np.empty(len(flat), np.int64)
    row[order] = np.arange(len(flat))
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=E + 1)[:E])])
    return offsets, np.where(key < E, row, -1 - row).reshape(ids.shape)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 128), (3, 2, 5), (31, 1, 1), (32, 8, 8), (64, 8, 128), (513, 3, 33),
                                   (512, 8, 1024), (513, 8, 1024), (1000, 7, 60), (4097, 1, 16), (5003, 4, 16),
                                   (16384, 8, 128), (20001, 32, 512)])
@pytest.mark.parametrize("dropped", [0.0, 0.2, 1.0])
def test_plan_is_the_stable_sort(T, k, E, dropped):
    from mxfp8_microscaled_precision_gb300 import mxq
    ids = _ids(T, k, E, 11 * T + E, dropped)
    offsets, rows = mxq.moe_plan(ids, E)
    want_off, want_rows = _plan64(ids, E)
    assert np.array_equal(offsets.cpu().numpy(), want_off)
    assert np.array_equal(rows.cpu().numpy(), want_rows)


def test_plan_of_one_expert_of_empty_ones_and_of_ids_out_of_range():
    from mxfp8_microscaled_precision_gb300 import mxq
    for ids, E in ((torch.full((700, 8), 17, dtype=torch.int32), 300),
                   (torch.full((9, 2), 5, dtype=torch.int32), 6),
                   (torch.tensor([[0, 4], [7, -5], [2 ** 31 - 1, 3]], dtype=torch.int32), 4)):
        ids = ids.cuda()
        offsets, rows = mxq.moe_plan(ids, E)
        want_off, want_rows = _plan64(ids, E)
        assert np.array_equal(offsets.cpu().numpy(), want_off) and np.array_equal(rows.cpu().numpy(), want_rows)
    offsets, rows = mxq.moe_plan(torch.empty(0, 8, dtype=torch.int32, device="cuda"), 12)
    assert offsets.tolist() == [0] * 13 and rows.shape == (0, 8)


SHAPES = [(1, 1, 1, 1), (1, 8, 128, 4096), (3, 2, 4, 7), (5, 8, 16, 513), (33, 4, 16, 1000), (64, 3, 8, 1026),
          (130, 8, 128, 2048), (17, 32, 64, 264), (9, 2, 4, 16384), (7, 5, 8, 9001)]


def _problem(T, k, E, H, dtype, seed, dropped=0.15):
    from mxfp8_microscaled_precision_gb300 import mxq
    g = torch.Generator().manual_seed(seed)
    offsets, rows = mxq.moe_plan(_ids(T, k, E, seed, dropped), E)
    w = torch.rand(T, k, generator=g).cuda()
    y = torch.randn(T * k, H, generator=g).to(dtype).cuda()
    x = torch.randn(T, H, generator=g).to(dtype).cuda()
    return offsets, rows, w, y, x


def _f64(t):
    return t.double().cpu().numpy()


def _places(rows):
    r = rows.cpu().numpy()
    return np.where(r < 0, -1 - r, r), r >= 0


def _close(got, ref, mag, eps, dtype, what):
    bound = eps * mag + (BF16 * np.abs(ref) if dtype == torch.bfloat16 else 0.0) + 1e-38
    assert np.all(np.abs(_f64(got) - ref) <= bound), (what, np.abs(_f64(got) - ref).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,E,H", SHAPES)
def test_dispatch_and_combine(T, k, E, H, dtype):
    from mxfp8_microscaled_precision_gb300 import mxq
    offsets, rows, w, y, x = _problem(T, k, E, H, dtype, 3 * T + H)
    at, kept = _places(rows)
    a = mxq.moe_dispatch(x, rows)
    want = torch.zeros_like(y)
    for j in range(k):
        want[torch.from_numpy(at[:, j]).cuda()] = x * torch.from_numpy(kept[:, j, None]).cuda()
    assert torch.equal(a, want)
    Y, W = _f64(y)[at] * kept[:, :, None], _f64(w)
    _close(mxq.moe_combine(y, rows, w), (Y * W[:, :, None]).sum(1), np.abs(Y * W[:, :, None]).sum(1), (k + 1) * EPS,
           dtype, "combine")
    _close(mxq.moe_combine(y, rows), Y.sum(1), np.abs(Y).sum(1), (k + 1) * EPS, dtype, "sum")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,E,H", SHAPES)
def test_combine_backward(T, k, E, H, dtype):
    from mxfp8_microscaled_precision_gb300 import mxq
    offsets, rows, w, y, dout = _problem(T, k, E, H, dtype, 5 * T + H)
    at, kept = _places(rows)
    dy, dw = mxq.moe_combine_backward(dout, y, rows, w)
    D, W = _f64(dout), _f64(w) * kept
    ref = np.empty((T * k, H))
    ref[at] = D[:, None, :] * W[:, :, None]
    _close(dy, ref, np.abs(ref), 2 * EPS, dtype, "dy")
    terms = D[:, None, :] * _f64(y)[at] * kept[:, :, None]
    _close(dw, terms.sum(2), np.abs(terms).sum(2), (H / 32 + 40) * EPS, torch.float32, "dweights")
    assert (dw.cpu().numpy()[~kept] == 0).all()


def test_gradients_against_differences():
    """combine is linear in y and in the weights, dispatch in x, so a difference of
    any step is the derivative: the kernels' gradients against differences of the kernels'
    own forward pass, all in small whole numbers that FP32 holds exactly."""
    from mxfp8_microscaled_precision_gb300 import mxq
    T, k, E, H = 6, 3, 4, 20
    g = torch.Generator().manual_seed(2)
    _, rows = mxq.moe_plan(_ids(T, k, E, 9, 0.2), E)

    def whole(*shape):
        return torch.randint(-4, 5, shape, generator=g).float().cuda()

    y, w, x, dout, da = whole(T * k, H), whole(T, k), whole(T, H), whole(T, H), whole(T * k, H)
    dy, dw = mxq.moe_combine_backward(dout, y, rows, w)
    dx = mxq.moe_combine(da, rows)

    def combined(yy, ww):
        return float((mxq.moe_combine(yy, rows, ww) * dout).sum())

    base = combined(y, w)
    for i in range(T * k):
        for h in (0, 7, 19):
            s = y.clone()
            s[i, h] += 1
            assert combined(s, w) - base == float(dy[i, h])
    for t in range(T):
        for j in range(k):
            s = w.clone()
            s[t, j] += 1
            assert combined(y, s) - base == float(dw[t, j])
        for h in (0, 19):
            s = x.clone()
            s[t, h] += 1
            assert float(((mxq.moe_dispatch(s, rows) - mxq.moe_dispatch(x, rows)) * da).sum()) == float(dx[t, h])


def test_dropped_rows_reach_nothing():
    """NaN in the rows behind the experts' (which the grouped products leave alone)
    and in the weights of dropped slots."""
    from mxfp8_microscaled_precision_gb300 import mxq
    for H in (64, 65):
        offsets, rows, w, y, x = _problem(40, 4, 8, H, torch.bfloat16, 77, 0.4)
        y[int(offsets[-1]):] = float("nan")
        w[rows < 0] = float("nan")
        out = mxq.moe_combine(y, rows, w)
        dy, dw = mxq.moe_combine_backward(x, y, rows, w)
        assert torch.isfinite(out).all() and torch.isfinite(dy).all() and torch.isfinite(dw).all()
        assert (dy[int(offsets[-1]):] == 0).all()
        assert (out[(rows < 0).all(1)] == 0).all() and bool((rows < 0).all(1).any())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,pad,shift", [(64, 8, 0), (64, 3, 0), (64, 8, 1), (65, 8, 0), (7, 2, 3), (1031, 2, 5),
                                         (4096, 1, 3)])
def test_strides_and_alignment(H, pad, shift, dtype):
    from mxfp8_microscaled_precision_gb300 import mxq
    T, k, E = 21, 4, 8
    offsets, rows, w, y, x = _problem(T, k, E, H, dtype, H + pad)

    def wide(t, fill):
        big = torch.full((t.shape[0], H + pad + shift), fill, dtype=dtype, device="cuda")
        big[:, shift:shift + H] = t
        return big, big[:, shift:shift + H]

    bx, vx = wide(x, float("nan"))
    by, vy = wide(y, float("nan"))
    for call, plain in ((lambda o: mxq.moe_dispatch(vx, rows, out=o), mxq.moe_dispatch(x, rows)),
                        (lambda o: mxq.moe_combine(vy, rows, w, out=o), mxq.moe_combine(y, rows, w)),
                        (lambda o: mxq.moe_combine_backward(vx, vy, rows, w, out=(o, None))[0],
                         mxq.moe_combine_backward(x, y, rows, w)[0])):
        big, view = wide(torch.zeros_like(plain), 7.0)
        got = call(view)
        assert torch.equal(got, plain)
        assert (big[:, :shift] == 7).all() and (big[:, shift + H:] == 7).all()
    # a tolerance for the dot product alone: another alignment may add in another order
    a, b = mxq.moe_combine_backward(vx, vy, rows, w)[1], mxq.moe_combine_backward(x, y, rows, w)[1]
    assert torch.all((a - b).abs() <= 2 * (H / 32 + 40) * EPS * H * 25)


def test_rows_past_two_to_the_31_elements():
    """T * k * H = 2.3e9 elements: offsets of the last rows do not fit 32 bits."""
    from mxfp8_microscaled_precision_gb300 import mxq
    T, k, E, H = 16385, 4, 8, 35072
    _, rows = mxq.moe_plan(_ids(T, k, E, 1), E)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = torch.arange(T, device="cuda") % 251
    x[:, -1] = torch.arange(T, device="cuda") % 241
    a = mxq.moe_dispatch(x, rows)
    for j in range(k):
        at = rows[:, j].long()
        assert torch.equal(a[at, 0], x[:, 0]) and torch.equal(a[at, H - 1], x[:, -1])
    w = torch.full((T, k), 0.25, device="cuda")
    out = mxq.moe_combine(a, rows, w)
    assert torch.equal(out, x)
    dy, dw = mxq.moe_combine_backward(x, a, rows, w)
    at = rows[:, k - 1].long()
    assert torch.equal(dy[at, H - 1].float(), x[:, -1].float() * 0.25)
    assert torch.equal(dw[:, 1].double(), (x[:, 0].double() ** 2 + x[:, -1].double() ** 2))


def test_no_tokens_same_answer_twice_and_refusals():
    from mxfp8_microscaled_precision_gb300 import mxq
    rows0 = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    assert mxq.moe_dispatch(torch.empty(0, 64, device="cuda"), rows0).shape == (0, 64)
    assert mxq.moe_combine(torch.empty(0, 64, device="cuda"), rows0).shape == (0, 64)
    offsets, rows, w, y, x = _problem(50, 4, 8, 200, torch.bfloat16, 4)
    one, two = mxq.moe_combine_backward(x, y, rows, w), mxq.moe_combine_backward(x, y, rows, w)
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    # rows that no plan gives are skipped, never followed
    far = torch.full_like(rows, 2 ** 31 - 1)
    assert (mxq.moe_combine(y, far, w) == 0).all()
    mxq.moe_dispatch(x, -far)
    for call in (lambda: mxq.moe_plan(torch.zeros(4, 2, dtype=torch.int64, device="cuda"), 4),
                 lambda: mxq.moe_plan(torch.zeros(4, 2, dtype=torch.int32, device="cuda"), 0),
                 lambda: mxq.moe_plan(torch.zeros(4, 2, dtype=torch.int32, device="cuda"), 1025),
                 lambda: mxq.moe_plan(torch.zeros(8, dtype=torch.int32, device="cuda"), 4),
                 lambda: mxq.moe_dispatch(x[:49], rows), lambda: mxq.moe_dispatch(x.half(), rows),
                 lambda: mxq.moe_dispatch(x, rows.long()), lambda: mxq.moe_dispatch(x.t(), rows),
                 lambda: mxq.moe_combine(y[:10], rows), lambda: mxq.moe_combine(y, rows, w.double()),
                 lambda: mxq.moe_combine_backward(x.float(), y, rows, w),
                 lambda: mxq.moe_dispatch(x, rows, out=torch.empty(3, 200, dtype=x.dtype, device="cuda"))):
        with pytest.raises(ValueError):
            call()
