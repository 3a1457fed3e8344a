"""Host-side checks of the operators around the GEMMs (no GPU needed): argument
validation rejects bad calls with the documented status before any CUDA work."""
import ctypes

import pytest

FAKE = ctypes.c_void_p(0x10000)        # aligned, never dereferenced
ODD = ctypes.c_void_p(0x10001)         # not on an element
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    from mxfp8_microscaled_precision_gb300 import build, mxq
    build.build()
    return mxq.lib()


def test_route_argument_errors(L):
    def r(logits=FAKE, dtype=1, T=4, E=64, ld=64, bias=None, mask=None, score=0, n=1, kept=1, gs=0, k=8, renorm=1,
          scale=1.0, ids=FAKE, w=FAKE):
        return L.mxq_route(logits, dtype, T, E, ld, bias, mask, score, n, kept, gs, k, renorm, scale, ids, w, None)
    assert r(T=0) == 0 and r(T=0, logits=None) == 0
    for bad in (dict(dtype=2), dict(T=-1), dict(E=0), dict(ld=63), dict(score=2), dict(n=0), dict(kept=0),
                dict(n=2, kept=3), dict(gs=2), dict(k=0), dict(k=65), dict(n=8, kept=1, k=9), dict(renorm=2),
                dict(scale=NAN), dict(scale=INF), dict(logits=None), dict(ids=None), dict(w=None), dict(logits=ODD),
                dict(bias=ODD), dict(ids=ODD)):
        assert r(**bad) == 1, bad
    for bad in (dict(E=1025, ld=1025), dict(k=33), dict(n=3), dict(n=64, kept=64), dict(T=1 << 31)):
        assert r(**bad) == 2, bad

    def b(dw=FAKE, ids=FAKE, logits=FAKE, dtype=1, T=4, E=64, ld=64, score=0, k=8, renorm=1, scale=1.0, out=FAKE, ldo=64):
        return L.mxq_route_backward(dw, ids, logits, dtype, T, E, ld, score, k, renorm, scale, out, ldo, None)
    assert b(T=0) == 0
    for bad in (dict(dtype=-1), dict(ldo=63), dict(k=0), dict(dw=None), dict(out=None), dict(out=ODD), dict(scale=NAN)):
        assert b(**bad) == 1, bad


def test_permute_argument_errors(L):
    p = L.mxq_moe_plan
    assert p(FAKE, 4, 2, 0, FAKE, FAKE, None) == 1 and p(FAKE, -1, 2, 8, FAKE, FAKE, None) == 1
    assert p(FAKE, 4, 2, 8, None, FAKE, None) == 1 and p(None, 4, 2, 8, FAKE, FAKE, None) == 1
    assert p(FAKE, 4, 2, 1025, FAKE, FAKE, None) == 2 and p(FAKE, 1 << 30, 2, 8, FAKE, FAKE, None) == 2
    d = L.mxq_moe_dispatch
    assert d(FAKE, 0, 0, 2, 64, 64, FAKE, FAKE, 64, None) == 0 and d(FAKE, 0, 4, 2, 0, 0, FAKE, FAKE, 0, None) == 0
    assert d(FAKE, 3, 4, 2, 64, 64, FAKE, FAKE, 64, None) == 1 and d(FAKE, 0, 4, 2, 64, 63, FAKE, FAKE, 64, None) == 1
    assert d(ODD, 0, 4, 2, 64, 64, FAKE, FAKE, 64, None) == 1 and d(FAKE, 0, 4, 2, 64, 64, None, FAKE, 64, None) == 1
    assert d(FAKE, 0, 4, 2, 1 << 24, 1 << 24, FAKE, FAKE, 1 << 24, None) == 2
    c = L.mxq_moe_combine
    assert c(FAKE, 1, 0, 2, 64, 64, FAKE, None, FAKE, 64, None) == 0
    assert c(FAKE, 1, 4, 2, 64, 64, FAKE, None, FAKE, 60, None) == 1 and c(None, 1, 4, 2, 64, 64, FAKE, None, FAKE, 64, None) == 1
    assert c(FAKE, 1, 4, 0, 64, 64, FAKE, None, FAKE, 64, None) == 1
    b = L.mxq_moe_combine_backward
    assert b(FAKE, FAKE, 0, 0, 2, 64, 64, 64, FAKE, FAKE, FAKE, 64, FAKE, None) == 0
    assert b(FAKE, FAKE, 0, 4, 2, 64, 64, 64, FAKE, None, FAKE, 64, FAKE, None) == 1
    assert b(FAKE, FAKE, 0, 4, 2, 64, 64, 64, FAKE, FAKE, FAKE, 64, None, None) == 1
    assert b(FAKE, FAKE, 0, 4, 2, 64, 32, 64, FAKE, FAKE, FAKE, 64, FAKE, None) == 1


def test_norm_argument_errors(L):
    n = L.mxq_layer_norm
    assert n(FAKE, 0, 0, 64, 64, None, None, 0, 1e-5, FAKE, 64, FAKE, FAKE, None) == 0
    for a in ((FAKE, 2, 4, 64, 64, None, None, 0, 1e-5, FAKE, 64, FAKE, FAKE, None),
              (FAKE, 0, 4, 64, 60, None, None, 0, 1e-5, FAKE, 64, FAKE, FAKE, None),
              (FAKE, 0, 4, 64, 64, None, None, 5, 1e-5, FAKE, 64, FAKE, FAKE, None),
              (FAKE, 0, 4, 64, 64, None, None, 0, -1.0, FAKE, 64, FAKE, FAKE, None),
              (FAKE, 0, 4, 64, 64, None, None, 0, NAN, FAKE, 64, FAKE, FAKE, None),
              (FAKE, 0, 4, 64, 64, None, None, 0, 1e-5, FAKE, 64, None, FAKE, None),
              (FAKE, 0, 4, 64, 64, ODD, None, 0, 1e-5, FAKE, 64, FAKE, FAKE, None)):
        assert n(*a) == 1, a
    assert n(FAKE, 0, 4, 1 << 24, 1 << 24, None, None, 0, 1e-5, FAKE, 1 << 24, FAKE, FAKE, None) == 2
    size = L.mxq_layer_norm_backward_workspace_size
    assert size(0, 64) == 0 and size(-1, 64) == 0 and size(10, 1 << 24) == 0
    assert 0 < size(1, 64) <= size(1000, 64) == size(10 ** 6, 64)
    b = L.mxq_layer_norm_backward
    Z = ctypes.c_size_t
    need = size(100, 64)
    assert b(FAKE, FAKE, 0, 100, 64, 64, 64, None, 0, FAKE, FAKE, FAKE, 64, FAKE, FAKE, FAKE, Z(need - 1), None) == 1
    assert b(FAKE, FAKE, 0, 100, 64, 64, 64, None, 0, FAKE, FAKE, FAKE, 64, FAKE, FAKE, None, Z(need), None) == 1
    assert b(FAKE, FAKE, 0, 100, 64, 64, 64, None, 0, FAKE, FAKE, FAKE, 32, FAKE, FAKE, FAKE, Z(need), None) == 1
    assert b(FAKE, FAKE, 0, 100, 64, 64, 64, None, 0, None, FAKE, FAKE, 64, FAKE, FAKE, FAKE, Z(need), None) == 1


def test_clip_argument_errors(L):
    from mxfp8_microscaled_precision_gb300 import mxq
    Z = ctypes.c_size_t
    size = L.mxq_grad_norm_workspace_size
    assert size(-1) == 0 and size(mxq.MAX_GRADS + 1) == 0 and 0 < size(0) <= size(mxq.MAX_GRADS)
    need = size(2)

    def call(f, count=2, grads=((0x10000, 0x20000, 8, 0), (0x30000, 0x40000, 8, 1)), norm=FAKE, ws=FAKE, bytes=need,
             args=(1.0, 1e-6)):
        d = (mxq.GradDesc * max(1, len(grads)))(*[mxq.GradDesc(*g) for g in grads])
        if f == "norm":
            return L.mxq_grad_norm(d, count, norm, ws, Z(bytes), None)
        return L.mxq_clip_grad_norm(d, count, *args, norm, ws, Z(bytes), None)
    for f in ("norm", "clip"):
        assert call(f, count=-1) == 1 and call(f, norm=None) == 1 and call(f, ws=None) == 1
        assert call(f, bytes=need - 1) == 1 and call(f, ws=ODD) == 1
        assert call(f, grads=((0x10000, 0x20000, 8, 2), (0x30000, 0x40000, 8, 1))) == 1      # dtype
        assert call(f, grads=((0x10000, 0x20000, -8, 0), (0x30000, 0x40000, 8, 1))) == 1     # size
        assert call(f, grads=((None, 0x20000, 8, 0), (0x30000, 0x40000, 8, 1))) == 1
        assert call(f, grads=((0x10001, 0x20000, 8, 0), (0x30000, 0x40000, 8, 1))) == 1
        assert call(f, count=mxq.MAX_GRADS + 1) == 2
    assert call("clip", grads=((0x10000, None, 8, 0), (0x30000, 0x40000, 8, 1))) == 1
    for args in ((-1.0, 1e-6), (NAN, 1e-6), (1.0, -1.0), (1.0, NAN), (1.0, INF)):
        assert call("clip", args=args) == 1


def test_python_calls_refuse_what_is_no_cuda_tensor(L):
    """The extension module checks its tensors before it allocates or calls anything."""
    import torch
    from mxfp8_microscaled_precision_gb300 import mxq
    x, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: mxq.route(x, 2), lambda: mxq.route(x, 2, score="relu"), lambda: mxq.route(x, 2, group_score="mean"),
                 lambda: mxq.route_backward(x, x, ids), lambda: mxq.moe_plan(ids, 4), lambda: mxq.moe_plan(ids[0], 4),
                 lambda: mxq.moe_dispatch(x, ids), lambda: mxq.moe_combine(x, ids), lambda: mxq.layer_norm(x),
                 lambda: mxq.moe_combine_backward(x, x, ids, x), lambda: mxq.layer_norm_backward(x, x, None, x[0], x[0]),
                 lambda: mxq.grad_norm([x]), lambda: mxq.clip_grad_norm([x], 1.0), lambda: mxq.clip_grad_norm([x], 1.0, out=[]),
                 lambda: mxq.grad_norm([x] * (mxq.MAX_GRADS + 1))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: mxq.route(None, 2), lambda: mxq.moe_plan([[1, 2]], 4), lambda: mxq.layer_norm("x"),
                 lambda: mxq.grad_norm([None]), lambda: mxq.clip_grad_norm([3], 1.0)):
        with pytest.raises(TypeError):
            call()
