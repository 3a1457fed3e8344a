"""Host-side checks of MXFP4 and of activations kept in 8 bits (no GPU needed): argument validation rejects bad calls
with the documented status before any CUDA work."""
import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(0x10000)        # aligned, never dereferenced
HALF = ctypes.c_void_p(0x10002)        # on a bf16 element
ODD = ctypes.c_void_p(0x10001)         # not on an element
BIG = 1 << 31


@pytest.fixture(scope="module")
def L():
    from mxfp8_microscaled_precision_gb300 import build, mxq
    build.build()
    return mxq.lib()


def test_quantization(L):
    def q(x=FAKE, dtype=0, batch=1, rows=4, cols=40, ld=40, stride=0, qr=FAKE, sr=FAKE, qc=FAKE, sc=FAKE, layout=1):
        return L.mxq_quant_mxfp4(x, dtype, batch, rows, cols, ld, stride, qr, sr, qc, sc, layout, None)
    assert q(rows=0, x=None) == 0 and q(cols=0, ld=0) == 0 and q(batch=0) == 0
    for bad in (dict(dtype=2), dict(layout=2), dict(batch=-1), dict(rows=-1), dict(cols=-1), dict(ld=39), dict(stride=-1),
                dict(x=None), dict(qr=None), dict(sr=None), dict(qc=None), dict(sc=None), dict(x=ODD), dict(x=HALF, dtype=1),
                dict(qr=HALF), dict(sr=HALF), dict(qc=HALF), dict(sc=HALF), dict(qr=None, sr=None, qc=None, sc=None)):
        assert q(**bad) == 1, bad
    for bad in (dict(batch=65536), dict(rows=BIG), dict(cols=BIG, ld=BIG), dict(rows=1 << 24, cols=1 << 24, ld=1 << 24),
                dict(batch=1024, rows=1 << 18, cols=1 << 18, ld=1 << 18)):
        assert q(**bad) == 2, bad

    def g(x=FAKE, dtype=1, rows=300, cols=40, ld=40, off=FAKE, G=4, cap=7, q=FAKE, s=FAKE):
        return L.mxq_quant_mxfp4_grouped(x, dtype, rows, cols, ld, off, G, cap, q, s, None)
    assert g(rows=0, cap=4) == 0
    for bad in (dict(dtype=-1), dict(rows=-1), dict(ld=39), dict(G=0), dict(cap=6), dict(x=None), dict(off=None), dict(q=None),
                dict(s=None), dict(x=HALF), dict(off=HALF), dict(q=HALF), dict(s=HALF)):
        assert g(**bad) == 1, bad
    assert g(G=1025, cap=2000) == 2 and g(rows=BIG, cap=BIG) == 2


def test_weight_gradients(L):
    def q(x=FAKE, dtype=0, rows=300, cols=40, ld=40, off=FAKE, G=4, cap=896, q=FAKE, s=FAKE):
        return L.mxq_quant_mxfp4_cols_grouped(x, dtype, rows, cols, ld, off, G, cap, q, s, None)
    assert q(rows=0, cap=512) == 0
    for bad in (dict(dtype=2), dict(rows=-1), dict(cols=-1), dict(ld=39), dict(G=0), dict(cap=768), dict(cap=-128), dict(x=None),
                dict(off=None), dict(q=None), dict(s=None), dict(x=ODD), dict(off=HALF), dict(q=HALF), dict(s=HALF)):
        assert q(**bad) == 1, bad
    assert q(G=1025, cap=1 << 20) == 2 and q(cap=900) == 2 and q(rows=BIG, cap=BIG) == 2

    def w(aq=FAKE, as_=FAKE, bq=FAKE, bs=FAKE, off=FAKE, G=4, rows=300, cap=896, M=24, N=40, y=FAKE, ldy=40):
        return L.mxq_grouped_gemm_mxfp4_wgrad(aq, as_, bq, bs, off, G, rows, cap, M, N, y, ldy, None)
    assert w(M=0) == 0 and w(N=0) == 0
    for bad in (dict(G=0), dict(rows=-1), dict(cap=-1), dict(cap=768), dict(M=-1), dict(N=-1), dict(ldy=39), dict(aq=None), dict(as_=None),
                dict(bq=None), dict(bs=None), dict(off=None), dict(y=None), dict(y=ODD), dict(off=HALF), dict(aq=HALF)):
        assert w(**bad) == 1, bad
    assert w(G=1025, cap=1 << 20) == 2 and w(cap=900) == 2 and w(M=1 << 30) == 2 and w(N=BIG, ldy=BIG) == 2


def test_values(L):
    def d(q=FAKE, s=FAKE, elem=0, rows=4, cols=40, ldq=40, lds=2, layout=0, out=FAKE, dtype=0, ldo=40):
        return L.mxq_dequant_1x32(q, s, elem, rows, cols, ldq, lds, layout, out, dtype, ldo, None)
    assert d(rows=0) == 0 and d(cols=0, ldq=0, lds=0, ldo=0) == 0
    for bad in (dict(elem=3), dict(elem=-1), dict(layout=5), dict(dtype=2), dict(rows=-1), dict(cols=-1), dict(ldq=39),
                dict(lds=1), dict(ldo=39), dict(q=None), dict(s=None), dict(out=None), dict(out=ODD), dict(out=HALF, dtype=1),
                dict(elem=2, ldq=31), dict(elem=2, ldq=34), dict(elem=2, q=HALF, ldq=32)):
        assert d(**bad) == 1, bad
    assert d(rows=BIG) == 2 and d(cols=1 << 24, ldq=1 << 24, lds=1 << 19, ldo=1 << 24) == 2


def test_products(L):
    def m(aq=FAKE, as_=FAKE, bq=FAKE, bs=FAKE, M=4, N=7, K=33, y=FAKE, ldy=7):
        return L.mxq_gemm_mxfp4(aq, as_, bq, bs, M, N, K, y, ldy, None)
    assert m(M=0) == 0 and m(N=0, ldy=0, y=None) == 0
    for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(ldy=6), dict(aq=None), dict(as_=None), dict(bq=None), dict(bs=None),
                dict(y=None), dict(aq=HALF), dict(as_=HALF), dict(bq=HALF), dict(bs=HALF), dict(y=ODD)):
        assert m(**bad) == 1, bad
    assert m(M=BIG) == 2 and m(N=BIG, ldy=BIG) == 2 and m(K=BIG) == 2

    def g(aq=FAKE, as_=FAKE, cap=7, bq=FAKE, bs=FAKE, off=FAKE, G=4, M=300, N=7, K=33, y=FAKE, ldy=7):
        return L.mxq_grouped_gemm_mxfp4(aq, as_, cap, bq, bs, off, G, M, N, K, y, ldy, None)
    assert g(M=0, cap=4) == 0
    for bad in (dict(M=-1), dict(N=-1), dict(K=0), dict(G=0), dict(ldy=6), dict(cap=6), dict(aq=None), dict(as_=None),
                dict(bq=None), dict(bs=None), dict(off=None), dict(y=None), dict(off=HALF), dict(bs=HALF), dict(y=ODD)):
        assert g(**bad) == 1, bad
    assert g(G=1025, cap=5000) == 2 and g(N=1 << 30, ldy=1 << 30) == 2 and g(M=BIG, cap=BIG) == 2


def test_activation(L):
    def f(z=FAKE, dtype=0, rows=4, inter=5, ldz=10, kind=0, gated=1, y=FAKE, ldy=5, q=FAKE, s=FAKE):
        return L.mxq_activation(z, dtype, rows, inter, ldz, kind, gated, y, ldy, q, s, None)
    assert f(rows=0) == 0 and f(inter=0, ldz=0, ldy=0, z=None) == 0
    for bad in (dict(dtype=2), dict(rows=-1), dict(inter=-1), dict(ldz=9), dict(gated=0, ldz=4), dict(kind=2), dict(gated=2),
                dict(ldy=4), dict(z=None), dict(y=None), dict(q=None), dict(s=None), dict(z=ODD), dict(z=HALF, dtype=1),
                dict(y=ODD), dict(q=HALF), dict(s=HALF)):
        assert f(**bad) == 1, bad
    assert f(rows=BIG) == 2 and f(inter=1 << 24, ldz=1 << 25, ldy=1 << 24) == 2

    def b(dy=FAKE, dtype=1, lddy=5, q=FAKE, s=FAKE, rows=4, inter=5, kind=1, gated=1, dz=FAKE, lddz=10, y=FAKE, ldy=5):
        return L.mxq_activation_backward(dy, dtype, lddy, q, s, rows, inter, kind, gated, dz, lddz, y, ldy, None)
    assert b(rows=0) == 0
    for bad in (dict(dtype=5), dict(lddy=4), dict(rows=-1), dict(kind=-1), dict(gated=-1), dict(lddz=9), dict(ldy=4),
                dict(dy=None), dict(q=None), dict(s=None), dict(dz=None), dict(dy=HALF), dict(dz=HALF), dict(y=HALF), dict(q=ODD)):
        assert b(**bad) == 1, bad
    assert b(rows=BIG) == 2


def test_python_calls_refuse_what_they_cannot_take(L):
    from mxfp8_microscaled_precision_gb300 import mxq
    x, u8, off = torch.zeros(4, 8), torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(3, dtype=torch.int64)
    for call in (lambda: mxq.quant_mxfp4(x), lambda: mxq.quant_mxfp4(x, layout="columns"), lambda: mxq.quant_mxfp4_grouped(x, off),
                 lambda: mxq.dequant_1x32(u8, u8, 8), lambda: mxq.dequant_1x32(u8, u8, 8, fmt="e3m2"),
                 lambda: mxq.dequant_1x32(u8, u8, 8, dtype=torch.float16), lambda: mxq.dequant_1x32(u8, u8, -1),
                 lambda: mxq.gemm_mxfp4(u8, u8, u8, u8, 4, 4, 32), lambda: mxq.gemm_mxfp4(u8, u8, u8, u8, 4, -4, 32),
                 lambda: mxq.gemm_mxfp4(u8, u8, u8, u8, 1 << 40, 4, 32), lambda: mxq.grouped_gemm_mxfp4(u8, u8, u8, u8, off, 4, 32),
                 lambda: mxq.activation(x), lambda: mxq.activation(x, kind="relu"), lambda: mxq.activation_backward(x, u8, u8),
                 lambda: mxq.activation_backward(x, u8, u8, kind="tanh")):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: mxq.quant_mxfp4(None), lambda: mxq.gemm_mxfp4(None, u8, u8, u8, 4, 4, 32), lambda: mxq.activation([1.0])):
        with pytest.raises(TypeError):
            call()


def test_the_bands_of_two_experts_never_meet():
    """The layout of mxq_quant_mxfp4_grouped: expert g starts at band floor(off[g]/128) + g, which leaves room for its
    ceil(n/128) bands before expert g + 1, and all fit ceil(rows/128) + G bands."""
    import random
    rng = random.Random(0)
    for _ in range(3000):
        G = rng.randint(1, 12)
        counts = [rng.choice([0, 1, 127, 128, 129, rng.randint(0, 700)]) for _ in range(G)]
        off = [sum(counts[:g]) for g in range(G + 1)]
        end = 0
        for g in range(G):
            first = off[g] // 128 + g
            assert first >= end
            end = first + -(-counts[g] // 128)
        assert end <= -(-(off[G] + rng.randint(0, 300)) // 128) + G
