"""MXFP4 and the activation on tensors of more than 2^31 elements: their last rows against a call on those rows alone,
byte by byte."""
import pytest
import torch

from _util import gpu_or_skip

pytestmark = pytest.mark.gpu

R, C, LAST = 135104, 16384, 256   # 2.2e9 elements; R a multiple of 128


@pytest.fixture(scope="module")
def x():
    gpu_or_skip()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    g = torch.Generator(device="cuda").manual_seed(0)
    t = torch.empty(R, C, dtype=torch.bfloat16, device="cuda")
    for part in t.split(8192):
        part.normal_(generator=g)
    yield t
    del t
    torch.cuda.empty_cache()


def test_quantization_and_values(x):
    from mxfp8_microscaled_precision_gb300 import mxq
    q, s, qc, sc = mxq.quant_mxfp4(x, layout="rowmajor")
    e, es, ec, esc = mxq.quant_mxfp4(x[-LAST:], layout="rowmajor")
    assert torch.equal(q[-LAST:], e) and torch.equal(s[-LAST:], es)
    assert torch.equal(qc[:, -LAST // 2:], ec) and torch.equal(sc[:, -LAST // 32:], esc)
    r, rs, _, _ = mxq.quant_mxfp4(x, col=False, layout="rowmajor")
    assert torch.equal(r, q) and torch.equal(rs, s)
    v = mxq.dequant_1x32(q, s, C, fmt="e2m1", layout="rowmajor")
    assert torch.equal(v[-LAST:], mxq.dequant_1x32(e, es, C, fmt="e2m1", layout="rowmajor"))


def test_activation(x):
    from mxfp8_microscaled_precision_gb300 import mxq
    y, q, s = mxq.activation(x)
    want = mxq.activation(x[-LAST:])
    assert all(torch.equal(a[-LAST:], b) for a, b in zip((y, q, s), want))
    dz, again = mxq.activation_backward(y, q, s)
    for a, b in zip((dz, again), mxq.activation_backward(want[0], *want[1:])):
        assert torch.equal(a[-LAST:], b)


@pytest.mark.parametrize("pad", [0, 3])
def test_products(x, pad):
    """Results of more than 2^31 elements, rows on 16 bytes and off them."""
    from mxfp8_microscaled_precision_gb300 import mxq
    N, K = C, 64
    a, w = x[:, :K].contiguous(), x[:N, :K].contiguous()
    qa, sa, _, _ = mxq.quant_mxfp4(a, col=False)
    qw, sw, _, _ = mxq.quant_mxfp4(w, col=False)
    y = torch.empty(R, N + pad, dtype=torch.bfloat16, device="cuda")[:, :N]
    mxq.gemm_mxfp4(qa, sa, qw, sw, R, N, K, out=y)
    last = mxq.quant_mxfp4(a[-LAST:], col=False)
    assert torch.equal(y[-LAST:], mxq.gemm_mxfp4(*last[:2], qw, sw, LAST, N, K))
    off = torch.tensor([0, 5, R - 60, R], device="cuda")
    y.zero_()
    stacked = torch.cat([w, w, w])
    qs, ss, _, _ = mxq.quant_mxfp4(stacked.view(3, N, K), col=False)
    mxq.grouped_gemm_mxfp4(*mxq.quant_mxfp4_grouped(a, off), qs, ss, off, N, K, out=y)
    assert torch.equal(y[-LAST:], mxq.gemm_mxfp4(*last[:2], qw, sw, LAST, N, K))
