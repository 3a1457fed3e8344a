"""How many digits the activation's FP32 results hold, from the middle to where they vanish, and what becomes of infinities.

Bounds, u = 2^-24 (a rounding of FP32), relative to the result unless said otherwise.  CUDA documents two units in the last place,
4u, for exp2f and for __fdividef; sums, products and divisions round by u.
Exponential: exp2f's 4u and the factor that follows, 5u: its argument's own error comes back in that factor.
SiLU: e = exp(-|g|) 5u, 1 + e 3.5u (e at most 1), its reciprocal 7.5u, times e 13.5u; f = g s 14.5u, times u or dy 15.5u.
The slope is s (1 + g s'), s' the other side's s: 13.5u of s, 14.5u of |g| s', the sum and the product u each, two more factors 2u:
32u of s (1 + |g| s').
GELU: t = k/(a + k) 5u; t P(t) changes by at most 3 times t's relative change, 15u; Horner's rule 3.4u, the factor t u, P itself 4.4e-8
or 0.8u; exp(-g^2/2) 5u; their product u.  Together 26.2u of the far side; of the near one, 1 - x with x at most 1/2, 27.2u.  f 28.2u,
times u 29.2u.  The slope, 27.2u of p, 7u of |g| bell and u of their sum, two more factors: 30.2u of p + |g| bell.
Where the exponential is below 2^-126 its steps are 2^-149, times |g| < 128: 2^-142; and results round by 2^-150."""
import math
import re
from pathlib import Path

import numpy as np
import pytest
import torch

from _util import gpu_or_skip

U = 2.0 ** -24
ABS = 2.0 ** -140
F_UNITS = {"silu": 16, "gelu": 30}      # rounded up: the products of roundings
SLOPE_UNITS = {"silu": 33, "gelu": 31}
SOURCE = Path(__file__).resolve().parents[1] / "mxfp8_microscaled_precision_gb300" / "csrc" / "act.cu"


def _parts(kind, g):
    """f, f' and the size that bounds f's slope's error, in 64 bits; the far side by erfc and not by 1 - erf."""
    if kind == "silu":
        p = 1.0 / (1.0 + torch.exp(-g))
        other = 1.0 / (1.0 + torch.exp(g))
        return g * p, p * (1 + g * other), p * (1 + g.abs() * other)
    p = 0.5 * torch.special.erfc(-g / math.sqrt(2))
    bell = torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    return g * p, p + g * bell, p + g.abs() * bell


def test_the_polynomial_is_as_near_as_its_comment_says():
    """The committed coefficients against exp(a^2/2) erfc(a / sqrt 2) / 2, and what the bounds above take from them."""
    from scipy.special import erfcx
    text = SOURCE.read_text()
    body = re.search(r"kP\[9\] = \{([^}]*)\}", text).group(1)
    c = np.array([np.float32(v.strip().rstrip("f")) for v in body.split(",")], np.float64)
    k = float(re.search(r"__fdividef\(([0-9.]+)f, a \+ \1f\)", text).group(1))
    stated = float(re.search(r"weighted towards equal relative errors: ([0-9.e-]+) at most", text).group(1))
    a = np.linspace(0, 15, 400001)
    t = k / (a + k)
    h = t * np.polynomial.polynomial.polyval(t, c)
    worst = np.abs(h / (erfcx(a / np.sqrt(2)) / 2) - 1).max()
    assert 0.9 * stated < worst <= stated <= 0.8 * U
    p, units = np.full_like(t, c[8]), np.zeros_like(t)
    for v in c[7::-1]:
        p = p * t + v
        units = units * t + np.abs(p)
    assert (units / np.abs(p)).max() < 3.4
    assert np.abs(np.gradient(np.log(h), np.log(t))).max() < 3.0


SPANS = {"silu": [(-103, -80), (-80, -70), (-70, -40), (-40, -20), (-20, -10), (-10, -4), (-4, -1), (-1, 1), (1, 4), (4, 20), (20, 103)],
         "gelu": [(-20, -14), (-14, -13), (-13, -12), (-12, -10), (-10, -8), (-8, -6), (-6, -4), (-4, -1), (-1, 1), (1, 4), (4, 20)]}


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [2048, 2047], ids=["vectors", "any"])
@pytest.mark.parametrize("kind,span", [(k, s) for k, spans in SPANS.items() for s in spans], ids=lambda v: v if isinstance(v, str) else f"{v[0]}to{v[1]}")
def test_fp32_results_hold_their_digits(kind, span, inter):
    gpu_or_skip()
    from mxfp8_microscaled_precision_gb300 import mxq
    gen = torch.Generator().manual_seed(inter)
    rows, units = 64, F_UNITS[kind] * U
    g = span[0] + (span[1] - span[0]) * torch.rand(rows, inter, generator=gen)
    u, dy = (1 + torch.rand(rows, inter, generator=gen) for _ in range(2))
    f, _, _ = _parts(kind, g.double())
    plain, _, _ = mxq.activation(g.cuda(), kind=kind, gated=False, checkpoint=False)
    assert bool(((plain.cpu().double() - f).abs() <= units * f.abs() + ABS).all())
    y, q, s = mxq.activation(torch.cat([g, u], 1).cuda(), kind=kind)
    want = f * u.double()
    assert bool(((y.cpu().double() - want).abs() <= units * want.abs() + ABS).all())
    # backward, at the values that the checkpoint stands for
    n = s.shape[1] // 2
    g8 = mxq.dequant_1x32(q[:, :inter], s[:, :n], inter, layout="rowmajor", dtype=torch.float32).cpu().double()
    u8 = mxq.dequant_1x32(q[:, inter:], s[:, n:], inter, layout="rowmajor", dtype=torch.float32).cpu().double()
    dz, again = (t.cpu().double() for t in mxq.activation_backward(dy.cuda(), q, s, kind=kind))
    f, slope, size = _parts(kind, g8)
    d = dy.double()
    assert bool(((again - f * u8).abs() <= units * (f * u8).abs() + ABS).all())
    assert bool(((dz[:, inter:] - d * f).abs() <= units * (d * f).abs() + ABS).all())
    assert bool(((dz[:, :inter] - d * u8 * slope).abs() <= SLOPE_UNITS[kind] * U * (d * u8 * size).abs() + 8 * ABS).all())
