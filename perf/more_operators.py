"""Cases of 4-bit microscaled values and of 8-bit activation checkpoints, next to the MXFP8 path of a training step:

  quant    a matrix in MXFP4 (E2M1 elements, one E8M0 scale per 32) along one or both axes, and the values it stands for
  gemm     the product of MXFP4 operands: a linear layer's forward pass or training step with the quantization
           of what is not kept in 4 bits, or the product of two operands that are
  grouped  the same for the experts of a mixture-of-experts layer, rows sorted by expert
  act      the (gated) activation between two products, its input kept in 8 bits (E4M3, one E8M0 scale per 32) for
           the backward pass

``run`` computes a case with elementary torch operations, or with the package's own kernels where
``own`` is true.  ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


def listed():
    return [
        # the rows of one decoding step, as the left operand of a product: latency alone
        dict(name="quant_decode", op="quant", rows=8, cols=4096, dtype="bf16", both=False),
        # a training step's activations for the forward pass and the weight gradient (the sweep's width 7168)
        dict(name="quant_train", op="quant", rows=16384, cols=7168, dtype="bf16", both=True),
        # no size a multiple of a group, in 32 bits
        dict(name="quant_odd", op="quant", rows=4099, cols=1111, dtype="f32", both=True),
        # one token through a layer whose weights are kept in 4 bits
        dict(name="gemm_decode", op="gemm", mode="forward", tokens=1, out=7168, inner=7168, dtype="bf16"),
        # a training step of a small layer of odd sizes: forward, input gradient, weight gradient
        dict(name="gemm_odd", op="gemm", mode="train", tokens=777, out=1003, inner=2085, dtype="f32"),
        # the linear layer's training step of the benchmark (8192 x 4096 x 4096)
        dict(name="gemm_train", op="gemm", mode="train", tokens=8192, out=4096, inner=4096, dtype="bf16"),
        # the largest product of the sweep, both operands in 4 bits already
        dict(name="gemm_large", op="gemm", mode="product", tokens=16384, out=16384, inner=16384, dtype="bf16"),
        # 8 sequences decode one token each: 64 rows to 128 experts, gate and up projection
        dict(name="grouped_decode", op="grouped", tokens=8, topk=8, experts=128, out=4096, inner=4096, dtype="bf16",
             dropped=0.0),
        # the forward pass of 16384 tokens through 128 experts
        dict(name="grouped_train", op="grouped", tokens=16384, topk=8, experts=128, out=4096, inner=4096, dtype="bf16",
             dropped=0.0),
        # the same decoding step's activation: nothing is kept
        dict(name="act_decode", op="act", rows=64, inter=2048, kind="silu", gated=True, dtype="bf16", keep=False),
        # a training step's, both directions
        dict(name="act_train", op="act", rows=131072, inter=2048, kind="silu", gated=True, dtype="bf16", keep=True),
        # an ungated one in 32 bits of a width that no group divides
        dict(name="act_odd", op="act", rows=4099, inter=1111, kind="gelu", gated=False, dtype="f32", keep=True),
    ]


def _spread(rng, lo, hi):
    """A size of [lo, hi], even over its logarithm: a power of two now and then, else odd."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    if rng.random() < 0.3:
        v = 2 ** round(math.log2(v))
    else:
        v = 2 * (int(v) // 2) + 1
    return max(lo, min(hi, int(v)))


def draw(rng):
    op = rng.choice(["quant", "gemm", "grouped", "act"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "quant":
        cols = _spread(rng, 32, 16384)
        return dict(op=op, rows=_spread(rng, 1, min(65536, 16384 * 7168 * 2 // (cols * SIZE[dtype]))), cols=cols, dtype=dtype,
                    both=rng.random() < 0.5)
    if op == "gemm":
        return dict(op=op, mode=rng.choice(["forward", "forward", "train", "product"]), tokens=_spread(rng, 1, 16384),
                    out=_spread(rng, 64, 8192), inner=_spread(rng, 64, 8192), dtype=dtype)
    if op == "grouped":
        experts, out, inner = _spread(rng, 2, 128), 8 * _spread(rng, 8, 512), 32 * _spread(rng, 2, 128)
        return dict(op=op, tokens=_spread(rng, 1, 16384), topk=rng.randint(1, min(8, experts)), experts=experts, out=out,
                    inner=inner, dtype="bf16", dropped=rng.choice([0.0, 0.1]))
    inter, gated = _spread(rng, 32, 8192), rng.random() < 0.6
    wide = inter * (2 if gated else 1) * SIZE[dtype]
    return dict(op=op, rows=_spread(rng, 1, min(131072, 131072 * 4096 * 2 // wide)), inter=inter, kind=rng.choice(["silu", "gelu"]),
                gated=gated, dtype=dtype, keep=rng.random() < 0.7)


# ---- the formats, by elementary operations in 32 bits -------------------------------------------------

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _groups(x):
    """x [..., K] in groups of 32 along its last axis, the last one filled up with zeros."""
    pad = -x.shape[-1] % 32
    if pad:
        x = torch.nn.functional.pad(x, (0, pad))
    return x.view(*x.shape[:-1], -1, 32)


def _exponent(g, most):
    """ceil(log2(amax / most)) of every group, most = 1.5 or 1.75 times a power of two; -127 at least."""
    m, e = torch.frexp(g.abs().amax(-1, keepdim=True))   # amax = m 2^e, m in [1/2, 1)
    ml, el = math.frexp(most)
    return torch.where(m == 0, -127, e - el + (m > ml)).clamp(min=-127)


def _fp4_codes(x):
    """(codes uint8 [..., groups, 32], exponents [..., groups, 1]) of x [..., K] in MXFP4."""
    g = _groups(x.float())
    e = _exponent(g, 6.0)
    a = torch.ldexp(g, -e)
    neg, a = torch.signbit(a), a.abs()
    code = torch.zeros(a.shape, dtype=torch.uint8, device=a.device)
    for at, even in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += a >= at if even else a > at   # a tie goes to the even code
    return code | (neg.to(torch.uint8) << 3), e


def _fp4_values(code, e, K):
    """FP32 [..., K] that codes and exponents stand for."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=code.device)
    return torch.ldexp(table[code.long()], e).flatten(-2)[..., :K]


def _fp4(x):
    """x as MXFP4 along its last axis holds it."""
    return _fp4_values(*_fp4_codes(x), x.shape[-1])


def _fp8(x):
    """x as MXFP8 (E4M3) along its last axis holds it."""
    g = _groups(x.float())
    e = _exponent(g, 448.0)
    a = torch.ldexp(g, -e)
    step = torch.frexp(a).exponent.clamp(min=-5) - 4   # 3 bits after the leading one, 2^-9 at least
    return torch.ldexp(torch.round(torch.ldexp(a, -step)), step + e).flatten(-2)[..., :x.shape[-1]]


def _packed(code):
    """Payload bytes [..., K/2] of codes [..., groups, 32]: two of them a byte, the first in the low half."""
    c = code.flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _tiled(s):
    """Scale codes [..., R, groups] in the order the tensor cores read them: 512-byte blocks of 128 rows x 4 groups,
    row r and group g of one at 16 (r % 32) + 4 (r / 32) + g; padded with zeros."""
    R, G = s.shape[-2:]
    s = torch.nn.functional.pad(s, (0, -G % 4, 0, -R % 128))
    s = s.view(*s.shape[:-2], s.shape[-2] // 128, 4, 32, s.shape[-1] // 4, 4)
    return s.movedim(-2, -4).transpose(-3, -2).reshape(-1).contiguous()


def _kept4(w):
    """A matrix [.., R, K] that a program keeps in 4 bits: payload, tiled scales, and plain ones."""
    code, e = _fp4_codes(w)
    plain = (e + 127).to(torch.uint8).squeeze(-1)
    return _packed(code), _tiled(plain), plain


def _restored4(q, s, K):
    """FP32 [R, K] of a payload and plain scales."""
    code = torch.stack((q & 15, q >> 4), -1).view(q.shape[0], -1, 32)
    return _fp4_values(code, s.to(torch.int32).unsqueeze(-1) - 127, K)


# ---- inputs ---------------------------------------------------------------------------------------

def _activations(gen, rows, cols, dtype):
    """Normal values with rare outliers 20 times as large, rows of different sizes."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x *= 0.5 + torch.rand(rows, 1, generator=gen, device="cuda")
    x[torch.rand(rows, cols, generator=gen, device="cuda") < 1e-3] *= 20
    return x.to(DTYPES[dtype])


def _expert_ids(gen, tokens, topk, experts):
    """topk different experts for each token, popular ones more often (Zipf 1.1)."""
    order = torch.argsort(torch.rand(experts, generator=gen, device="cuda"))
    popularity = -1.1 * torch.log(torch.arange(1, experts + 1, device="cuda").float())[order]
    gumbel = -torch.log(-torch.log(torch.rand(tokens, experts, generator=gen, device="cuda").clamp_(1e-20, 1 - 1e-6)))
    return torch.topk(popularity + gumbel, topk, dim=1).indices


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    state, op = dict(case), case["op"]
    dtype = DTYPES[case["dtype"]]
    if op == "quant":
        state["x"] = _activations(gen, case["rows"], case["cols"], case["dtype"])
    elif op == "gemm":
        M, N, K = case["tokens"], case["out"], case["inner"]
        x, w = _activations(gen, M, K, case["dtype"]), (0.02 * randn(N, K)).to(dtype)
        state["x"], state["w"] = x, w
        if case["mode"] == "train":
            state["dy"] = (1e-3 * randn(M, N)).to(dtype)
        else:   # the weights are kept in 4 bits, of a product both operands are
            state["w"] = _kept4(w)
            if case["mode"] == "product":
                state["x"] = _kept4(x)
    elif op == "grouped":
        T, k, E, N, K = (case[n] for n in ("tokens", "topk", "experts", "out", "inner"))
        ids = _expert_ids(gen, T, k, E)
        live = torch.rand(T, generator=gen, device="cuda") >= case["dropped"]
        count = torch.bincount(ids[live].reshape(-1), minlength=E)
        state["offsets"] = torch.nn.functional.pad(torch.cumsum(count, 0), (1, 0))
        state["host_offsets"] = state["offsets"].tolist()
        state["x"] = _activations(gen, T * k, K, case["dtype"])
        kept = [_kept4((0.02 * randn(N, K)).to(dtype)) for _ in range(E)]
        state["w"] = torch.cat([q for q, _, _ in kept]), torch.cat([t for _, t, _ in kept]), torch.cat([s for _, _, s in kept])
        state["y"] = torch.zeros(T * k, N, dtype=torch.bfloat16, device="cuda")   # rows behind the last expert's stay as they are
    else:
        M, C = case["rows"], case["inter"] * (2 if case["gated"] else 1)
        state["z"] = (1.5 * randn(M, C) * (0.5 + torch.rand(M, 1, generator=gen, device="cuda"))).to(dtype)
        if case["keep"]:
            state["dy"] = (1e-3 * randn(M, case["inter"])).to(dtype)
    return state


# ---- one pass ---------------------------------------------------------------------------------------

def run(state):
    return {"quant": _quant, "gemm": _gemm, "grouped": _grouped, "act": _act}[state["op"]](state)


def _quant(s):
    x, R, C = s["x"], s["rows"], s["cols"]
    if own:
        from mxfp8_microscaled_precision_gb300 import mxq
        q, sc, qt, sct = mxq.quant_mxfp4(x, col=s["both"])
        row = mxq.dequant_1x32(q, sc, C, fmt="e2m1")
        return [row, mxq.dequant_1x32(qt, sct, R, fmt="e2m1")] if s["both"] else [row]
    out = [_fp4(x)] + ([_fp4(x.t().contiguous())] if s["both"] else [])
    return [v.to(torch.bfloat16) for v in out]


def _gemm(s):
    M, N, K = s["tokens"], s["out"], s["inner"]
    if own:
        from mxfp8_microscaled_precision_gb300 import mxq
        if s["mode"] == "train":
            x, xs, xt, xts = mxq.quant_mxfp4(s["x"])
            w, ws, wt, wts = mxq.quant_mxfp4(s["w"])
            d, ds, dt, dts = mxq.quant_mxfp4(s["dy"])
            return {"y": mxq.gemm_mxfp4(x, xs, w, ws, M, N, K), "dx": mxq.gemm_mxfp4(d, ds, wt, wts, M, K, N),
                    "dw": mxq.gemm_mxfp4(dt, dts, xt, xts, N, K, M)}
        x, xs = s["x"][:2] if s["mode"] == "product" else mxq.quant_mxfp4(s["x"], col=False)[:2]
        return {"y": mxq.gemm_mxfp4(x, xs, *s["w"][:2], M, N, K)}
    bf16 = torch.bfloat16
    if s["mode"] == "train":
        x, w, dy = s["x"], s["w"], s["dy"]
        t = lambda v: _fp4(v.t().contiguous())  # noqa: E731
        return {"y": (_fp4(x) @ _fp4(w).t()).to(bf16), "dx": (_fp4(dy) @ t(w).t()).to(bf16), "dw": (t(dy) @ t(x).t()).to(bf16)}
    x = _restored4(s["x"][0], s["x"][2], K) if s["mode"] == "product" else _fp4(s["x"])
    return {"y": (x @ _restored4(s["w"][0], s["w"][2], K).t()).to(bf16)}


def _grouped(s):
    N, K = s["out"], s["inner"]
    if own:
        from mxfp8_microscaled_precision_gb300 import mxq
        x, xs = mxq.quant_mxfp4_grouped(s["x"], s["offsets"])
        return mxq.grouped_gemm_mxfp4(x, xs, *s["w"][:2], s["offsets"], N, K, out=s["y"])
    q, _, sc = s["w"]
    at = s["host_offsets"]
    for g in range(s["experts"]):   # one product after the other: no elementary operation takes experts of different sizes
        if at[g + 1] > at[g]:
            w = _restored4(q[g * N:(g + 1) * N], sc[g * N:(g + 1) * N], K)
            s["y"][at[g]:at[g + 1]] = (_fp4(s["x"][at[g]:at[g + 1]]) @ w.t()).to(torch.bfloat16)
    return s["y"]


def _act_parts(s, z):
    """f(g), f'(g) and u (1 without a gate) of z in 32 bits."""
    z = z.float()
    g, u = (z[:, :s["inter"]], z[:, s["inter"]:]) if s["gated"] else (z, torch.ones((), device=z.device))
    if s["kind"] == "silu":
        sig = 1.0 / (1.0 + torch.exp(-g))
        return g * sig, sig * (1.0 + g * (1.0 - sig)), u
    cdf = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
    return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi)), u


def _act(s):
    if own:
        from mxfp8_microscaled_precision_gb300 import mxq
        kw = dict(kind=s["kind"], gated=s["gated"])
        y, q, sc = mxq.activation(s["z"], checkpoint=s["keep"], **kw)
        if not s["keep"]:
            return {"y": y}
        dz, again = mxq.activation_backward(s["dy"], q, sc, **kw)
        return {"y": y, "dz": dz, "again": again}
    z, dtype = s["z"], s["z"].dtype
    f, _, u = _act_parts(s, z)
    out = {"y": (f * u).to(dtype)}
    if s["keep"]:
        I = s["inter"]
        kept = torch.cat([_fp8(z[:, :I]), _fp8(z[:, I:])], 1) if s["gated"] else _fp8(z)
        f, df, u = _act_parts(s, kept)
        dy = s["dy"].float()
        dz = torch.cat([dy * u * df, dy * f], 1) if s["gated"] else dy * df
        out.update(dz=dz.to(dtype), again=(f * u).to(dtype))
    return out


# ---- what a pass has to move and compute ---------------------------------------------------------------

def _bytes4(R, K):
    """Payload and scales of a matrix [R, K] in MXFP4."""
    return R * -(-K // 32) * 17


def work(case):
    op = case["op"]
    b = SIZE[case["dtype"]]
    if op == "quant":   # x read, the copies and the values they stand for written
        R, C = case["rows"], case["cols"]
        return {"bytes": R * C * b + _bytes4(R, C) + 2 * R * C + (_bytes4(C, R) + 2 * R * C if case["both"] else 0),
                "flops": 4 * R * C * (2 if case["both"] else 1)}
    if op == "gemm":
        M, N, K = case["tokens"], case["out"], case["inner"]
        if case["mode"] == "train":
            return {"bytes": (M * K + N * K + M * N) * (b + 2), "flops": 6 * M * N * K}
        x = _bytes4(M, K) if case["mode"] == "product" else M * K * b
        return {"bytes": x + _bytes4(N, K) + 2 * M * N, "flops": 2 * M * N * K}
    if op == "grouped":
        rows, N, K, E = case["tokens"] * case["topk"], case["out"], case["inner"], case["experts"]
        # the weights of the experts that have rows, each once: as many as Zipf's law lets one expect
        zipf = [(i + 1) ** -1.1 for i in range(E)]
        hit = sum(1 - (1 - min(1.0, case["topk"] * p / sum(zipf))) ** case["tokens"] for p in zipf)
        return {"bytes": rows * K * b + round(hit * _bytes4(N, K)) + 2 * rows * N, "flops": 2 * rows * N * K}
    M, C = case["rows"], case["inter"] * (2 if case["gated"] else 1)
    size, flops = M * (C + case["inter"]) * b, 10 * M * case["inter"]
    if case["keep"]:   # the checkpoint written and read; dy read, dz and the output written again
        size += 2 * M * -(-C // 32) * 33 + M * (C + 2 * case["inter"]) * b
        flops *= 3
    return {"bytes": size, "flops": flops}


# ---- the definitions in 64 bits ---------------------------------------------------------------------------

def _two(e):
    """2^e in 64 bits, exactly: a power function is off by a rounding for some of them."""
    return (e.long() + 1023 << 52).view(torch.float64)


def _held(x, most, grid):
    """x [R, K] in groups of 32 along a row, each a grid's nearest values times the least power of two that holds the group:
    the definition, value by value.  grid(a): the nearest value to each a >= 0, ties to the even one."""
    R, K = x.shape
    x = torch.nn.functional.pad(x.double(), (0, -K % 32)).view(R, -1, 32)
    top = x.abs().max(2, keepdim=True).values
    e = torch.ceil(torch.log2(top / most)).clamp(min=-127)   # within one of it; then exactly
    e = torch.where(most * _two(e - 1) >= top, e - 1, e)
    e = torch.where(most * _two(e) < top, e + 1, e)
    two = _two(e.clamp(min=-127))
    return (torch.sign(x) * grid((x / two).abs()) * two).view(R, -1)[:, :K]


def _grid4(a):
    # below 2 the values are halves, below 4 wholes, then 4 and 6
    return torch.where(a <= 2, torch.round(2 * a) / 2, torch.where(a <= 4, torch.round(a), 2 * torch.round(a / 2)))


def _grid8(a):
    unit = _two(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.round(a / unit) * unit   # no 32-bit value is so near a power of two that its logarithm rounds there


def _hold4(x, rows=2048):
    return torch.cat([_held(p, 6.0, _grid4) for p in x.split(rows)])


def _hold8(x, rows=16384):
    return torch.cat([_held(p, 448.0, _grid8) for p in x.split(rows)])


def _value4(q, s, K):
    """64-bit values of a payload [R, K/2] with plain scales, rows at a time."""
    table = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device=q.device) / 2
    out = []
    for p, c in zip(q.split(2048), s.split(2048)):
        both = torch.stack([p % 16, p // 16], 2).view(p.shape[0], -1).long()
        v = table[both % 8] * (1 - 2 * (both // 8))
        out.append((v.view(p.shape[0], -1, 32) * _two(c.long() - 127)[:, :, None]).view(p.shape[0], -1)[:, :K])
    return torch.cat(out)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "quant":
        out = [_hold4(s["x"])]
        return out + [_hold4(s["x"].t())] if case["both"] else out
    if op == "gemm":
        K = case["inner"]
        if case["mode"] == "train":
            x, w, dy = s["x"], s["w"], s["dy"]
            return {"y": torch.einsum("mk,nk->mn", _hold4(x), _hold4(w)), "dx": torch.einsum("mn,kn->mk", _hold4(dy), _hold4(w.t())),
                    "dw": torch.einsum("nm,km->nk", _hold4(dy.t()), _hold4(x.t()))}
        x = _value4(s["x"][0], s["x"][2], K) if case["mode"] == "product" else _hold4(s["x"])
        return {"y": torch.einsum("mk,nk->mn", x, _value4(s["w"][0], s["w"][2], K))}
    if op == "grouped":
        N, K, at, out = case["out"], case["inner"], s["host_offsets"], s["y"].double()
        for g in range(case["experts"]):
            if at[g + 1] > at[g]:
                w = _value4(s["w"][0][g * N:(g + 1) * N], s["w"][2][g * N:(g + 1) * N], K)
                out[at[g]:at[g + 1]] = torch.einsum("mk,nk->mn", _hold4(s["x"][at[g]:at[g + 1]]), w)
        return out
    def parts(z):
        g, u = (z[:, :case["inter"]], z[:, case["inter"]:]) if case["gated"] else (z, torch.ones((), dtype=z.dtype, device=z.device))
        if case["kind"] == "silu":
            p = torch.sigmoid(g)
            return g * p, p + g * p * torch.sigmoid(-g), u
        p = 0.5 * torch.special.erfc(-g / math.sqrt(2.0))
        return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2.0 * math.pi), u
    f, _, u = parts(s["z"].double())
    out = {"y": f * u}
    if case["keep"]:
        I, z = case["inter"], s["z"]
        f, df, u = parts(torch.cat([_hold8(z[:, :I]), _hold8(z[:, I:])], 1) if case["gated"] else _hold8(z))
        dy = s["dy"].double()
        out.update(dz=torch.cat([dy * u * df, dy * f], 1) if case["gated"] else dy * df, again=f * u)
    return out
