"""The activation between two products and its gradients from an input kept in 8 bits, on the GPU against 64 bits.

Tolerances, u = 2^-24 (a rounding of FP32): the exponential and erfc of the CUDA library are off by at most 2 and 4 units
of 2u, the other operations by u each, so f(g) by at most 24 u |f(g)| (its argument is rounded once: that is up to
|g|^2 u of erfc's and |g| u of exp's value: + 2 g^2 u), f'(g) by as much of the sum of its terms' sizes.  A
product adds u for each factor.  BF16 results are off by 2^-8 of themselves; below 2^-126 nothing is held.
The checkpoint is compared byte by byte."""
import math

import numpy as np
import pytest
import torch

import _fp4
from _util import gpu_or_skip

U = 2.0 ** -24


def _parts(z, inter, kind, gated):
    """f, f', u, and the sizes that bound f's and f's slope's errors, in 64 bits."""
    z = torch.from_numpy(z)
    g, u = (z[:, :inter], z[:, inter:]) if gated else (z, torch.ones(1, dtype=torch.float64))
    if kind == "silu":
        p = torch.sigmoid(g)
        f, df, size = g * p, p * (1 + g * torch.sigmoid(-g)), p * (1 + g.abs() * (1 + torch.sigmoid(-g)))
    else:
        p = 0.5 * torch.special.erfc(-g / math.sqrt(2))
        bell = torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        f, df, size = g * p, p + g * bell, p + g.abs() * bell
    return f, df, u, (24 + 2 * g * g) * U * f.abs(), (24 + 2 * g * g) * U * size


def test_the_slopes_are_those_of_differences():
    """The formulas against central differences in 64 bits (error h^2 / 6 f''' and 2^-52 / h)."""
    g = np.linspace(-9, 9, 4001)[None]
    for kind in ("silu", "gelu"):
        h = 1e-4
        up, down = _parts(g + h, g.size, kind, False)[0], _parts(g - h, g.size, kind, False)[0]
        assert float(((up - down) / (2 * h) - _parts(g, g.size, kind, False)[1]).abs().max()) < 1e-7


CASES = [(1, 1), (1, 8), (2, 31), (3, 32), (5, 33), (64, 2048), (1, 4096), (100, 100), (33, 1111), (257, 96), (40, 520), (9, 8192)]


def _input(rows, cols, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    z = 3 * torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-4, 3, (rows, 1), generator=g).float())
    if rows > 2:
        z[1] = 0.0
        z[2] = torch.linspace(-120, 120, cols)
    return z.to(dtype)


def _near(got, want, bound):
    err = (got.detach().double().cpu() - want).abs()
    if got.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (want.abs() + bound)
    assert bool((err <= bound + 2.0 ** -126).all()), float((err - bound).max())


def _kept(z, inter, gated):
    """(payload, scales, values) of the checkpoint."""
    halves = [z[:, :inter], z[:, inter:]] if gated else [z]
    made = [_fp4.quantize(h, "e4m3") for h in halves]
    return (np.concatenate([c[:, :inter] for c, _ in made], 1), np.concatenate([s for _, s in made], 1),
            np.concatenate([_fp4.values(c, s, inter, "e4m3") for c, s in made], 1))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
@pytest.mark.parametrize("rows,inter", CASES)
def test_both_directions(rows, inter, gated, kind, dtype):
    gpu_or_skip()
    from mxfp8_microscaled_precision_gb300 import mxq
    cols = inter * (2 if gated else 1)
    z = _input(rows, cols, dtype, rows + inter)
    y, q, s = mxq.activation(z.cuda(), kind=kind, gated=gated)
    f, _, u, ef, _ = _parts(_fp4.f64(z), inter, kind, gated)
    _near(y, f * u, (ef + 2 * U * f.abs()) * u.abs())
    payload, scales, values = _kept(_fp4.f64(z), inter, gated)
    assert np.array_equal(q.cpu().numpy(), payload) and np.array_equal(s.cpu().numpy(), scales)
    alone = mxq.activation(z.cuda(), kind=kind, gated=gated, checkpoint=False)
    assert alone[1] is None and alone[2] is None and torch.equal(alone[0], y)
    dy = torch.randn(rows, inter, generator=torch.Generator().manual_seed(5)).to(dtype)
    dz, again = mxq.activation_backward(dy.cuda(), q, s, kind=kind, gated=gated)
    f, df, u, ef, edf = _parts(values, inter, kind, gated)
    _near(again, f * u, (ef + 2 * U * f.abs()) * u.abs())
    d = dy.double()
    _near(dz[:, :inter], d * u * df, (d * u).abs() * (edf + 3 * U * df.abs()))
    if gated:
        _near(dz[:, inter:], d * f, d.abs() * (ef + 2 * U * f.abs()))
    only, none = mxq.activation_backward(dy.cuda(), q, s, kind=kind, gated=gated, output=False)
    assert none is None and torch.equal(only, dz)
    # the checkpoint's halves are payloads as any other
    groups = -(-inter // 32)
    back = mxq.dequant_1x32(q[:, :inter], s[:, :groups], inter, layout="rowmajor", dtype=torch.float32)
    assert np.array_equal(_fp4.f64(back), values[:, :inter])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("off,pad", [(0, 0), (0, 8), (1, 0), (3, 5), (2, 1)])
@pytest.mark.parametrize("inter", [64, 77])
def test_rows_that_start_anywhere(inter, off, pad, dtype):
    gpu_or_skip()
    from mxfp8_microscaled_precision_gb300 import mxq

    def view(rows, cols, fill):
        flat = torch.full((off + rows * (cols + pad) + 40,), fill, dtype=dtype, device="cuda")
        return flat, flat[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]

    z, dy = _input(37, 2 * inter, dtype, 3).cuda(), torch.randn(37, inter, device="cuda").to(dtype)
    want = mxq.activation(z)
    grads = mxq.activation_backward(dy, *want[1:])
    vz, vdy = view(37, 2 * inter, float("nan"))[1].copy_(z), view(37, inter, float("nan"))[1].copy_(dy)
    (fy, vy), (fdz, vdz), (fa, va) = view(37, inter, 9.0), view(37, 2 * inter, 9.0), view(37, inter, 9.0)
    y, q, s = mxq.activation(vz, out=(vy, None, None))
    assert y is vy and all(torch.equal(a, b) for a, b in zip((y, q, s), want))
    dz, again = mxq.activation_backward(vdy, q, s, out=(vdz, va))
    assert dz is vdz and again is va and torch.equal(dz, grads[0]) and torch.equal(again, grads[1])
    for flat, v in ((fy, vy), (fdz, vdz), (fa, va)):
        inside = torch.zeros_like(flat, dtype=torch.bool)
        inside[off:off + 37 * (v.shape[1] + pad)].view(37, v.shape[1] + pad)[:, :v.shape[1]] = True
        assert bool((flat[~inside] == 9).all())


@pytest.mark.gpu
def test_nan_and_infinity_reach_their_own_group_only():
    gpu_or_skip()
    from mxfp8_microscaled_precision_gb300 import mxq
    z = torch.randn(4, 200, device="cuda")
    z[1, 3], z[2, 150], z[3, 99] = float("nan"), float("inf"), -float("inf")
    y, q, s = mxq.activation(z)
    hit = torch.zeros(4, 100, dtype=torch.bool)
    hit[1, 3] = True
    assert torch.equal(y.isnan().cpu(), hit) and math.isinf(float(y[2, 50])) and float(y[3, 99]) == 0.0 or y[3, 99].isnan()
    dz, again = mxq.activation_backward(torch.ones(4, 100, device="cuda"), q, s)
    want = torch.zeros(4, 200, dtype=torch.bool)
    want[1, 0:32] = want[1, 100:132] = True     # g's group: both gradients need g
    want[2, 32:64] = True                       # u's group (columns 32 .. 63 of u): dg needs u, du does not
    want[3, 96:100] = want[3, 196:200] = True
    assert torch.equal(dz.isnan().cpu(), want)
    assert bool((s[1, 0] == 255) & (s[2, 5] == 255) & (s[3, 3] == 255)) and int((s == 255).sum()) == 3


@pytest.mark.gpu
def test_empty_streams_and_graphs():
    gpu_or_skip()
    from mxfp8_microscaled_precision_gb300 import mxq
    y, q, s = mxq.activation(torch.empty(0, 64, device="cuda"))
    assert y.shape == (0, 32) and q.shape == (0, 64) and s.shape == (0, 2)
    assert mxq.activation_backward(y, q, s)[0].shape == (0, 64)
    z, dy = torch.randn(50, 300, device="cuda").bfloat16(), torch.randn(50, 150, device="cuda").bfloat16()

    def step():
        y, q, s = mxq.activation(z)
        return (y, *mxq.activation_backward(dy, q, s))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, step()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in range(2):
        z.copy_(torch.randn(50, 300, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(held, step()))


@pytest.mark.gpu
def test_refusals():
    gpu_or_skip()
    from mxfp8_microscaled_precision_gb300 import mxq
    z = torch.randn(4, 65, device="cuda")
    y, q, s = mxq.activation(z, gated=False)
    for call in (lambda: mxq.activation(z), lambda: mxq.activation(z.half(), gated=False), lambda: mxq.activation(z.t(), gated=False),
                 lambda: mxq.activation_backward(y, q, s), lambda: mxq.activation_backward(y, q[:, :-1], s, gated=False),
                 lambda: mxq.activation_backward(y, q, s[:3], gated=False),
                 lambda: mxq.activation(z, gated=False, out=(y[:, 1:], None, None)),
                 lambda: mxq.activation(z, gated=False, checkpoint=False, out=(None, q, s)),
                 lambda: mxq.activation_backward(y, q, s, gated=False, output=False, out=(None, y))):
        with pytest.raises(ValueError):
            call()
