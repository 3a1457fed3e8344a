"""The norm over all gradients and clipping on the GPU (mxq.grad_norm,
clip_grad_norm) against numpy in 64 bits.

Tolerance of the norm: squares and their sums within a thread's share are rounded to
FP32 (at most n = elements / 150000 + 200 additions in a row), the rest is FP64: relative
(n + 2) 2^-24, halved by the root.  A scaled gradient adds the rounding of the factor
and of the product: (n + 8) 2^-24 relative, BF16 another 2^-8 (half a unit in the last place)."""
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


def _grads(sizes, seed, std=1e-3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(std * torch.randn(n, generator=g, device="cuda")).to(d) for n, d in sizes]


def _norm64(grads):
    return math.sqrt(sum(float((t.double() ** 2).sum()) for t in grads))


def _check(grads, max_norm, outs, norm, eps=1e-6):
    n = sum(g.numel() for g in grads) / 150000 + 200
    ref = _norm64(grads)
    assert abs(float(norm) - ref) <= (n + 2) / 2 * EPS * ref
    c = min(1.0, max_norm / (ref + eps))
    for g, o in zip(grads, outs):
        want = g.double() * c
        tol = (n + 8) * EPS + (BF16 if g.dtype == torch.bfloat16 else 0.0)
        assert o.dtype == g.dtype and torch.all((o.double() - want).abs() <= tol * want.abs() + 1e-40)


B, F = torch.bfloat16, torch.float32
LISTS = [
    [(1, B)],
    [(1, F)],
    [(7, B), (9, F), (8, B), (0, F), (16, B), (3, F)],
    [(4096, F), (512 * 512, B), (33, B)],
    [(16384, B), (16385, B), (8192, F), (8193, F), (8191, F)],
    [(1000003, B), (700001, F)],
    [(40_000_000, B), (20_000_000, F)],
    [(i % 97, (B, F)[i % 2]) for i in range(1500)],       # more tensors than one launch takes
    [(3000 + 17 * i, (B, F)[i % 3 == 0]) for i in range(1024)],
    [(3000 + 17 * i, (B, F)[i % 3 == 0]) for i in range(65)],
]


@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: f"{len(s)}x{s[0][0]}")
@pytest.mark.parametrize("max_norm", [1e-2, 1e9])
def test_clip_against_64_bits(sizes, max_norm):
    from mxfp8_microscaled_precision_gb300 import mxq
    grads = _grads(sizes, len(sizes))
    keep = [g.clone() for g in grads]
    norm, outs = mxq.clip_grad_norm(grads, max_norm)
    _check(grads, max_norm, outs, norm)
    assert all(torch.equal(a, b) for a, b in zip(keep, grads))
    assert float(mxq.grad_norm(grads)) == float(norm)
    again, outs2 = mxq.clip_grad_norm(grads, max_norm, out=grads)      # in place
    assert float(again) == float(norm) and all(a is b for a, b in zip(outs2, grads))
    assert all(torch.equal(a, b) for a, b in zip(outs, grads))


def test_views_of_a_flat_buffer_at_any_element():
    """Tensors that start at any element, outputs aligned alike and differently; what
    lies between them is left alone."""
    from mxfp8_microscaled_precision_gb300 import mxq
    for dtype in (B, F):
        sizes = [5, 1, 8, 4099, 13, 65536, 2, 31]
        for shift in (0, 1, 3, 5):
            flat = torch.full((sum(sizes) + 8 * len(sizes) + 8,), 7.0, dtype=dtype, device="cuda")
            to = torch.full_like(flat, 9.0)
            at, grads, outs, inside = 1, [], [], torch.zeros_like(flat, dtype=torch.bool)
            for n in sizes:
                grads.append(flat[at:at + n])
                grads[-1].normal_()
                outs.append(to[at + shift:at + shift + n])
                inside[at + shift:at + shift + n] = True
                at += n + 3
            norm, _ = mxq.clip_grad_norm(grads, 0.5, out=outs)
            _check(grads, 0.5, outs, norm)
            assert (to[~inside] == 9).all()


def test_bad_values_and_no_gradients():
    from mxfp8_microscaled_precision_gb300 import mxq
    assert float(mxq.grad_norm([])) == 0.0
    norm, out = mxq.clip_grad_norm([], 1.0)
    assert float(norm) == 0.0 and out == []
    z = [torch.zeros(100, device="cuda"), torch.empty(0, dtype=B, device="cuda")]
    norm, out = mxq.clip_grad_norm(z, 1.0)
    assert float(norm) == 0.0 and (out[0] == 0).all()
    g = _grads([(1000, B), (1000, F)], 3, std=1.0)
    norm, out = mxq.clip_grad_norm(g, 0.0)
    assert all((o == 0).all() for o in out)
    norm, out = mxq.clip_grad_norm(g, math.inf)
    assert all(torch.equal(a, b) for a, b in zip(out, g))
    bad = [t.clone() for t in g]
    bad[0][17] = math.nan
    norm, out = mxq.clip_grad_norm(bad, 1.0)
    assert math.isnan(float(norm)) and all(torch.isnan(o).all() for o in out)
    bad[0][17] = math.inf
    norm, out = mxq.clip_grad_norm(bad, 1.0)
    assert math.isinf(float(norm)) and math.isnan(float(out[0][17])) and (out[1] == 0).all()


def test_a_tensor_past_two_to_the_32_bytes():
    from mxfp8_microscaled_precision_gb300 import mxq
    n = (1 << 31) + 4097
    g = torch.zeros(n, dtype=B, device="cuda")
    g[0] = 3.0
    g[n - 1] = 4.0
    norm, (o,) = mxq.clip_grad_norm([g], 2.5, eps=0.0, out=[g])
    assert float(norm) == 5.0 and float(o[0]) == 1.5 and float(o[n - 1]) == 2.0 and float(o[n // 2]) == 0.0


def test_same_answer_on_every_call_and_another_stream():
    from mxfp8_microscaled_precision_gb300 import mxq
    g = _grads([(3_000_001, B), (999, F), (1_000_000, F)], 12)
    want = mxq.grad_norm(g)
    assert all(torch.equal(mxq.grad_norm(g), want) for _ in range(5))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = mxq.grad_norm(g)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


def test_refusals():
    from mxfp8_microscaled_precision_gb300 import mxq
    g = torch.ones(16, device="cuda")
    for call in (lambda: mxq.grad_norm([g.double()]), lambda: mxq.grad_norm([g.cpu()]),
                 lambda: mxq.grad_norm([torch.ones(4, 4, device="cuda").t()[:, :2]]),
                 lambda: mxq.clip_grad_norm([g], -1.0), lambda: mxq.clip_grad_norm([g], math.nan),
                 lambda: mxq.clip_grad_norm([g], 1.0, eps=-1.0), lambda: mxq.clip_grad_norm([g], 1.0, eps=math.inf),
                 lambda: mxq.clip_grad_norm([g], 1.0, out=[]),
                 lambda: mxq.clip_grad_norm([g], 1.0, out=[g.bfloat16()]),
                 lambda: mxq.clip_grad_norm([g], 1.0, out=[g[:8]])):
        with pytest.raises(ValueError):
            call()
