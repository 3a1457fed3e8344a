"""Routing to experts on the GPU (mxq.route, mxq.route_backward) against the
definition in 64 bits, one token at a time in numpy.

Tolerance of the weights: a score is exp of a difference rounded to FP32
(relative error |x - max| 2^-24), an exponential of at most 2 ulp, a sum of at
most 32 + 5 rounded additions and a division, and renormalising adds a sum of 32 and a
division: (2 |x - max| + 128) 2^-24 covers both.  A gradient is a sum of up to 32
such terms, so its absolute error is bounded by that factor times 4 sum |terms|.
BF16 results add half a unit in the last place, 2^-8 relative.
"""
import math

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


def _scores(x, score):
    """64-bit scores of one token's logits."""
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-x))
    m = x.max()
    e = np.exp(x - (m if np.isfinite(m) else 0.0))
    return e / e.sum() if e.sum() > 0 else e


def _choice(x, bias, score, n_group, topk_group, group_score):
    """(choice values with -inf for experts that are out, scores) of one token."""
    s = _scores(x, score)
    c = x.copy() if bias is None else np.where(x == -math.inf, -math.inf, s + bias)
    if n_group > 1:
        by = s if bias is None and group_score == "top2sum" else c
        by = np.where(c == -math.inf, -math.inf, by).reshape(n_group, -1)
        top = np.sort(by, axis=1)[:, ::-1]
        g = top[:, 0].copy()
        if group_score == "top2sum" and top.shape[1] > 1:
            g = np.where(top[:, 1] > -math.inf, top[:, 0] + top[:, 1], top[:, 0])
        best = sorted(range(n_group), key=lambda i: (-g[i], i))[:topk_group]
        stays = np.isin(np.arange(n_group), best).repeat(len(x) // n_group)
        c = np.where(stays, c, -math.inf)
    return c, s


def _weights(s, ids, renorm, scale):
    chosen = np.where(ids >= 0, s[np.maximum(ids, 0)], 0.0)
    w = scale * chosen
    return w / (chosen.sum() + 1e-20) if renorm else w


def _gradient(x, ids, dw, score, renorm, scale):
    """(dlogits, bound's sum of |terms|) of one token in 64 bits."""
    s = _scores(x, score)
    ok = ids >= 0
    at = ids[ok]
    dw = dw[ok]
    if not ok.any():
        return np.zeros_like(x), np.zeros_like(x)
    ds = np.zeros_like(x)
    mag = np.zeros_like(x)
    total = s[at].sum() + 1e-20
    if renorm:
        ds[at] = (scale * dw - (dw * scale * s[at] / total).sum()) / total
        mag[at] = scale * (np.abs(dw) + (np.abs(dw) * s[at] / total).sum()) / total
    else:
        ds[at] = scale * dw
        mag[at] = scale * np.abs(dw)
    if score == "sigmoid":
        slope = s * _scores(-x, "sigmoid")
        return ds * slope, mag * slope
    return s * (ds - (ds * s).sum()), s * (mag + (mag * s).sum())


def _check_forward(logits, ids, w, bias, score, n_group, topk_group, group_score, renorm, scale, mask=None):
    X = logits.double().cpu().numpy()
    B = None if bias is None else bias.double().cpu().numpy()
    I, Wt = ids.cpu().numpy(), w.double().cpu().numpy()
    for t in range(X.shape[0]):
        if mask is not None and not bool(mask[t]):
            assert (I[t] == -1).all() and (Wt[t] == 0).all()
            continue
        c, s = _choice(X[t], B, score, n_group, topk_group, group_score)
        want = np.sort(c[c > -math.inf])[::-1][:I.shape[1]]
        got = I[t]
        n = len(want)
        assert (got[n:] == -1).all() and (got[:n] >= 0).all(), (t, got, n)
        assert len(set(got[:n])) == n and (got[:n] < X.shape[1]).all()
        if B is None:   # the logits themselves are compared: exact, ties to the lowest expert
            order = sorted(np.flatnonzero(c > -math.inf), key=lambda e: (-c[e], e))[:n]
            assert got[:n].tolist() == [int(e) for e in order], t
        else:           # values that differ by less than the scores' rounding may change places
            assert np.all(np.abs(c[got[:n]] - want) <= 4e-6), t
        ref = _weights(s, got, renorm, scale)
        fin = X[t][X[t] > -math.inf]
        span = 2 * (fin.max() - fin.min()) + 2 * np.abs(fin).max() if len(fin) else 0.0
        assert np.all(np.abs(Wt[t] - ref) <= (span + 128) * EPS * np.abs(ref) + 1e-37), t


CASES = [  # E, topk, score, bias, n_group, topk_group, group_score, renorm, scale
    (1, 1, "softmax", False, 1, 1, "max", True, 1.0),
    (5, 5, "sigmoid", False, 1, 1, "max", True, 1.0),
    (8, 2, "softmax", False, 1, 1, "max", False, 1.0),
    (32, 4, "softmax", True, 1, 1, "max", True, 2.5),
    (33, 32, "sigmoid", True, 1, 1, "max", True, 1.0),
    (60, 6, "softmax", False, 6, 2, "max", True, 1.0),
    (60, 7, "sigmoid", True, 12, 5, "top2sum", True, 2.5),
    (64, 1, "sigmoid", False, 1, 1, "max", False, 1.0),
    (128, 8, "softmax", False, 1, 1, "max", True, 1.0),
    (130, 8, "softmax", False, 1, 1, "max", True, 1.0),
    (256, 8, "sigmoid", True, 8, 4, "top2sum", True, 2.5),
    (256, 8, "sigmoid", False, 8, 4, "top2sum", False, 1.0),
    (255, 9, "softmax", True, 3, 2, "top2sum", True, 1.0),
    (32, 3, "sigmoid", True, 32, 3, "top2sum", True, 1.0),     # groups of one expert
    (512, 16, "softmax", False, 16, 3, "max", False, 1.0),
    (1000, 10, "sigmoid", True, 1, 1, "max", True, 1.0),
    (1024, 32, "softmax", False, 32, 32, "max", True, 1.0),
]


def _inputs(T, E, dtype, seed, bias):
    g = torch.Generator().manual_seed(seed)
    x = (2 * torch.randn(T, E, generator=g)).to(dtype).cuda()
    b = (torch.randint(-30, 31, (E,), generator=g) / 1000).float().cuda() if bias else None
    return x, b


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_route_against_64_bits(case, dtype):
    from mxfp8_microscaled_precision_gb300 import mxq
    E, k, score, bias, n, kept, gs, renorm, scale = case
    for T in (1, 4, 131):
        x, b = _inputs(T, E, dtype, 100 * E + T, bias)
        ids, w = mxq.route(x, k, score, b, n, kept, gs, renorm, scale)
        _check_forward(x, ids, w, b, score, n, kept, gs, renorm, scale)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_route_backward_against_64_bits(case, dtype):
    from mxfp8_microscaled_precision_gb300 import mxq
    E, k, score, bias, n, kept, gs, renorm, scale = case
    T = 37
    x, b = _inputs(T, E, dtype, 7 * E, bias)
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    mask[3] = mask[36] = False
    x[3] = math.nan
    ids, _ = mxq.route(x, k, score, b, n, kept, gs, renorm, scale, token_mask=mask)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(E)).cuda()
    dx = mxq.route_backward(dw, x, ids, score, renorm, scale)
    assert dx.dtype == dtype and dx.shape == x.shape
    X, I, D, G = (v.double().cpu().numpy() for v in (x, ids, dw, dx))
    for t in range(T):
        if not bool(mask[t]):
            assert (G[t] == 0).all()
            continue
        ref, mag = _gradient(X[t], I[t].astype(int), D[t], score, renorm, scale)
        span = 4 * np.abs(X[t]).max()
        bound = 4 * (span + 128) * EPS * mag + 1e-37
        if dtype == torch.bfloat16:
            bound = bound + BF16 * np.abs(ref)
        assert np.all(np.abs(G[t] - ref) <= bound), (t, np.abs(G[t] - ref).max())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_against_differences(score, renorm):
    """Central differences of sum(dw * w) in 64 bits with the choice held: step h
    leaves an error of h^2 (third derivatives, below 10 here) and 1e-16 / h; the kernel's own
    bound of the test above, 4 (32 + 128) 2^-24 times at most 2 scale |dw|, is below 1e-4 of scale |dw|."""
    from mxfp8_microscaled_precision_gb300 import mxq
    T, E, k, scale, h = 5, 24, 4, 2.5, 1e-5
    x, _ = _inputs(T, E, torch.float32, 5, False)
    ids, _ = mxq.route(x, k, score, renorm=renorm, scale=scale)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(6)).cuda()
    dx = mxq.route_backward(dw, x, ids, score, renorm, scale).double().cpu().numpy()
    X, I, D = x.double().cpu().numpy(), ids.cpu().numpy(), dw.double().cpu().numpy()
    for t in range(T):
        for e in range(E):
            step = np.zeros(E)
            step[e] = h
            f = [(D[t] * _weights(_scores(X[t] + sgn * step, score), I[t], renorm, scale)).sum() for sgn in (1, -1)]
            assert abs((f[0] - f[1]) / (2 * h) - dx[t, e]) <= 1e-8 + 1e-4 * np.abs(D[t]).max() * scale


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("scale", [1.0, 2.0])
def test_one_expert_with_all_the_weight_has_no_gradient(score, scale):
    """top 1, renormalised: the weight is the scale whatever the logits are.  With a power of two every step is
    exact (s / s = 1, two equal products), so the gradient is 0 and not a rounding of it."""
    from mxfp8_microscaled_precision_gb300 import mxq
    gen = torch.Generator(device="cuda").manual_seed(7)
    x = 3.0 * torch.randn(1000, 72, generator=gen, device="cuda")
    dw = torch.randn(1000, 1, generator=gen, device="cuda")
    ids, w = mxq.route(x, 1, score=score, renorm=True, scale=scale)
    assert (w == scale).all()
    assert (mxq.route_backward(dw, x, ids, score=score, renorm=True, scale=scale) == 0).all()


def test_ties_go_to_the_lowest_expert():
    from mxfp8_microscaled_precision_gb300 import mxq
    for E in (40, 128, 700):
        x = torch.zeros(3, E, device="cuda")
        x[1] = -0.0
        x[1, 7] = 0.0
        x[2, 5::9] = 1.0
        for score in ("softmax", "sigmoid"):
            for bias in (None, torch.zeros(E, device="cuda")):
                ids, w = mxq.route(x, 4, score, bias)
                assert ids.tolist() == [[0, 1, 2, 3], [0, 1, 2, 3], [5, 14, 23, 32]], (E, score)
                assert torch.allclose(w, torch.full_like(w, 0.25), rtol=4 * EPS, atol=0)
    # equal groups: the lowest ones stay
    ids, _ = mxq.route(torch.zeros(1, 40, device="cuda"), 6, "softmax", n_group=8, topk_group=2)
    assert ids.tolist() == [[0, 1, 2, 3, 4, 5]]


def test_masked_experts_and_rows():
    """-inf logits and biases take experts out; a row with none left gets -1 and 0;
    the lowest finite value stays eligible."""
    from mxfp8_microscaled_precision_gb300 import mxq
    for dtype in (torch.float32, torch.bfloat16):
        for score in ("softmax", "sigmoid"):
            x = torch.full((5, 48), -math.inf, dtype=dtype, device="cuda")
            x[1, 40] = 0.5
            x[2, [3, 33, 9]] = torch.tensor([-1.0, 2.0, 0.0], dtype=dtype, device="cuda")
            x[3] = torch.finfo(dtype).min
            x[4, :24] = torch.finfo(dtype).min
            ids, w = mxq.route(x, 4, score)
            assert ids.tolist() == [[-1] * 4, [40, -1, -1, -1], [33, 9, 3, -1], [0, 1, 2, 3], [0, 1, 2, 3]]
            assert torch.isfinite(w).all() and (w[0] == 0).all() and (w[1, 1:] == 0).all()
            assert w[1, 0] == 1.0 and abs(float(w[2].sum()) - 1) < 1e-6
            g = mxq.route_backward(torch.ones(5, 4, device="cuda"), x, ids, score)
            assert torch.isfinite(g).all() and (g[0] == 0).all()
            b = torch.zeros(48, device="cuda")
            b[33] = -math.inf
            assert mxq.route(x, 4, score, b)[0][2].tolist() == [9, 3, -1, -1]
            ids, _ = mxq.route(x, 4, score, n_group=4, topk_group=2, group_score="top2sum")
            assert ids[2, :2].tolist() == [33, 9] or ids[2, :2].tolist() == [9, 3]
            assert ids[0].tolist() == [-1] * 4


def test_nan_and_inf_stay_in_their_rows():
    from mxfp8_microscaled_precision_gb300 import mxq
    x = torch.randn(6, 64, generator=torch.Generator().manual_seed(1)).cuda()
    clean, wc = mxq.route(x, 3, "sigmoid")
    y = x.clone()
    y[1] = math.nan
    y[3, 10] = math.nan
    y[4, 20] = math.inf
    for score in ("softmax", "sigmoid"):
        ids, w = mxq.route(y, 3, score)
        assert (ids >= 0).all() and (ids < 64).all() and all(len(set(r)) == 3 for r in ids.tolist())
        assert ids[1].tolist() == [0, 1, 2] and torch.isnan(w[1]).all()
        assert ids[4, 0] == 20
        assert torch.equal(ids[[0, 2, 5]], clean[[0, 2, 5]]) and torch.isfinite(w[[0, 2, 5]]).all()
    ids, w = mxq.route(y, 3, "sigmoid")
    assert 10 not in ids[3].tolist() and torch.isfinite(w[3]).all()
    # padding tokens: what stands in them reaches nothing
    mask = torch.tensor([1, 0, 1, 0, 0, 1], dtype=torch.uint8, device="cuda")
    ids, w = mxq.route(y, 3, "softmax", token_mask=mask)
    assert (ids[mask == 0] == -1).all() and (w[mask == 0] == 0).all()
    g = mxq.route_backward(torch.ones(6, 3, device="cuda"), y, ids, "softmax")
    assert (g[mask == 0] == 0).all() and torch.isfinite(g).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [31, 64, 128, 129])
def test_strides_and_alignment(E, dtype):
    from mxfp8_microscaled_precision_gb300 import mxq
    T, k = 19, 5
    wide = torch.full((T, E + 13), math.nan, dtype=dtype, device="cuda")
    x, b = _inputs(T, E, dtype, 3, True)
    wide[:, 3:3 + E] = x
    view = wide[:, 3:3 + E]
    for kw in (dict(), dict(bias=b, score="sigmoid")):
        a, c = mxq.route(x, k, **kw), mxq.route(view, k, **kw)
        assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])
        score = kw.get("score", "softmax")
        dw = torch.randn(T, k, device="cuda")
        to = torch.full((T, E + 9), 7.0, dtype=dtype, device="cuda")
        got = mxq.route_backward(dw, view, a[0], score, out=to[:, 5:5 + E])
        assert torch.equal(got, mxq.route_backward(dw, x, a[0], score))
        assert (to[:, :5] == 7).all() and (to[:, 5 + E:] == 7).all()


def test_no_tokens_and_another_stream():
    from mxfp8_microscaled_precision_gb300 import mxq
    ids, w = mxq.route(torch.empty(0, 16, device="cuda"), 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)
    assert mxq.route_backward(w, torch.empty(0, 16, device="cuda"), ids).shape == (0, 16)
    x = torch.randn(4096, 128, device="cuda")
    want = mxq.route(x, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = mxq.route(x, 8)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_refusals():
    from mxfp8_microscaled_precision_gb300 import mxq
    x = torch.randn(4, 64, device="cuda")
    for bad in (dict(topk=65), dict(topk=0), dict(topk=33), dict(topk=4, score="relu"), dict(topk=4, n_group=3),
                dict(topk=4, n_group=4, topk_group=5), dict(topk=40, n_group=4, topk_group=2),
                dict(topk=4, n_group=64, topk_group=64), dict(topk=4, scale=math.nan),
                dict(topk=4, bias=torch.zeros(63, device="cuda")), dict(topk=4, group_score="min"),
                dict(topk=4, bias=torch.zeros(64, device="cuda", dtype=torch.bfloat16)),
                dict(topk=4, token_mask=torch.ones(5, dtype=torch.bool, device="cuda")),
                dict(topk=4, token_mask=torch.ones(4, device="cuda"))):
        with pytest.raises(ValueError):
            mxq.route(x, **bad)
    for bad in (x.half(), x.cpu(), x[0], x.t(), torch.randn(2, 1025, device="cuda")):
        with pytest.raises(ValueError):
            mxq.route(bad, 1)
    ids, w = mxq.route(x, 4)
    with pytest.raises(ValueError):
        mxq.route_backward(w, x, ids.long())
    with pytest.raises(ValueError):
        mxq.route_backward(w[:, :3], x, ids)
