"""Cases of the operators around the experts' products of an MXFP8 mixture-of-experts training step:

  route    scores of the experts, groups, the k best, their weights; backward to the logits
  permute  the plan (expert order of the rows, offsets), rows into expert order, the weighted sum back; backward
  norm     layer norm, forward and backward with the gradients of weight and bias
  clip     the norm over all gradients, and the gradients scaled to a largest norm

``run`` computes a case with elementary torch operations, or with the package's own kernels where
``own`` is true.  ``exact`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
RENORM_EPS = 1e-20
NORM_EPS = 1e-5
CLIP_EPS = 1e-6


def listed():
    return [
        # one decoding step of a few sequences: latency alone
        dict(name="route_decode", op="route", tokens=4, experts=128, topk=8, score="softmax", bias=False, groups=1,
             kept_groups=1, group_score="max", scale=1.0, dtype="f32", masked=0.0, backward=False),
        # a training step's router: 16384 tokens, 128 experts, top 8 (the routing of the moe workloads)
        dict(name="route_train", op="route", tokens=16384, experts=128, topk=8, score="softmax", bias=False, groups=1,
             kept_groups=1, group_score="max", scale=1.0, dtype="f32", masked=0.0, backward=True),
        # sigmoid scores balanced by a bias, limited to 4 of 8 groups, padded sequences, a ragged batch
        dict(name="route_grouped", op="route", tokens=8191, experts=256, topk=8, score="sigmoid", bias=True, groups=8,
             kept_groups=4, group_score="top2sum", scale=2.5, dtype="bf16", masked=0.05, backward=True),
        # one decoding step through 128 experts
        dict(name="permute_decode", op="permute", tokens=8, hidden=4096, experts=128, topk=8, dtype="bf16", dropped=0.0,
             backward=False),
        # a training step: the rows of 16384 tokens to 128 experts and back
        dict(name="permute_train", op="permute", tokens=16384, hidden=4096, experts=128, topk=8, dtype="bf16", dropped=0.0,
             backward=False),
        # its backward pass at another width, few experts, a ragged batch with padding tokens
        dict(name="permute_backward", op="permute", tokens=10007, hidden=7168, experts=16, topk=4, dtype="bf16",
             dropped=0.1, backward=True),
        # one decoding step
        dict(name="norm_decode", op="norm", rows=8, cols=4096, dtype="bf16", wdtype="bf16", backward=False),
        # a training step, both directions
        dict(name="norm_train", op="norm", rows=16384, cols=7168, dtype="bf16", wdtype="bf16", backward=True),
        # a width that no vector divides, in 32 bits
        dict(name="norm_odd", op="norm", rows=4099, cols=1111, dtype="f32", wdtype="f32", backward=True),
        # a small dense layer: a few small gradients
        dict(name="clip_small", op="clip", tensors=6, largest=512 * 512, f32_part=0.3, packed=False, sizes=1,
             max_norm=0.5),
        # the gradients of 16 experts (gate and up 4096 x 4096, down 4096 x 2048) with their router and norms
        dict(name="clip_experts", op="clip", tensors=36, largest=4096 * 4096, f32_part=0.1, packed=False, sizes=2,
             max_norm=1.0),
        # many gradients of odd sizes packed without gaps
        dict(name="clip_ragged", op="clip", tensors=300, largest=1000003, f32_part=0.5, packed=True, sizes=3,
             max_norm=0.5),
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
    op = rng.choice(["route", "permute", "norm", "clip"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "route":
        score = rng.choice(["softmax", "sigmoid"])
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _spread(rng, 8, 512 // groups)
        kept = rng.randint(1, groups)
        # a bias and sums of scores go with sigmoid scores, the maximum of a group with softmax
        return dict(op=op, tokens=_spread(rng, 1, 32768), experts=experts,
                    topk=rng.randint(1, min(16, experts // groups * kept)), score=score, bias=score == "sigmoid" and rng.random() < 0.7,
                    groups=groups, kept_groups=kept, group_score="top2sum" if score == "sigmoid" and rng.random() < 0.7 else "max",
                    scale=rng.choice([1.0, 2.5]), dtype=dtype, masked=rng.choice([0.0, 0.05]), backward=rng.random() < 0.5)
    if op == "permute":
        hidden = rng.choice([8 * _spread(rng, 8, 1024), _spread(rng, 64, 8192)])
        experts = _spread(rng, 2, 512)
        topk = rng.randint(1, min(8, experts))
        most = 16384 * 8 * 4096 * 4 // 3 // (hidden * topk * SIZE[dtype])
        return dict(op=op, tokens=_spread(rng, 1, min(32768, most)), hidden=hidden, experts=experts, topk=topk, dtype=dtype,
                    dropped=rng.choice([0.0, 0.1]), backward=rng.random() < 0.5)
    if op == "norm":
        cols = rng.choice([8 * _spread(rng, 8, 2048), _spread(rng, 64, 16384)])
        most = 16384 * 7168 * 2 // (cols * SIZE[dtype])
        return dict(op=op, rows=_spread(rng, 1, min(32768, most)), cols=cols, dtype=dtype,
                    wdtype=rng.choice([dtype, "f32"]), backward=rng.random() < 0.5)
    tensors = _spread(rng, 1, 400)
    return dict(op=op, tensors=tensors, largest=_spread(rng, 64, min(2 ** 24, 2 ** 28 // tensors)),
                f32_part=rng.choice([0.0, 0.3, 1.0]), packed=rng.random() < 0.5, sizes=rng.randint(4, 1 << 20),
                max_norm=rng.choice([0.5, 1.0, 1e9]))


# ---- inputs ---------------------------------------------------------------------------------------

def _clip_sizes(case):
    """(elements, dtype) of every gradient: a third matrices of the largest size or a half of it, the others spread below."""
    rng = random.Random(case["sizes"])
    most, got = case["largest"], []
    for i in range(case["tensors"]):
        if case["packed"]:
            n = _spread(rng, 1, most)
        else:
            n = most if i % 3 == 0 else most // 2 if i % 3 == 1 and most > 1 else max(1, most // 1024)
        got.append((n, "f32" if rng.random() < case["f32_part"] else "bf16"))
    return got


def _places(case):
    """{dtype: (elements of its flat buffer, [(start, elements)])}: gaps up to 256 bytes unless packed."""
    out = {}
    for d in ("bf16", "f32"):
        at, spans, step = 0, [], 1 if case["packed"] else 256 // SIZE[d]
        for n, kind in _clip_sizes(case):
            if kind == d:
                spans.append((at, n))
                at = -(-(at + n) // step) * step
        out[d] = (at, spans)
    return out


def _logits(gen, tokens, experts):
    """What a router says in training: a spread per token and a standing preference for some experts."""
    popular = 0.7 * torch.randn(experts, generator=gen, device="cuda")
    return 1.3 * torch.randn(tokens, experts, generator=gen, device="cuda") + popular


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rand = lambda *shape: torch.rand(*shape, generator=gen, device="cuda")  # noqa: E731
    randn = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    state = dict(case)
    op = case["op"]
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["topk"]
        state["logits"] = _logits(gen, T, E).to(DTYPES[case["dtype"]])
        # a bias moves by steps of a thousandth towards balance
        state["bias"] = torch.round(20 * randn(E)) / 1000 if case["bias"] else None
        state["mask"] = rand(T) >= case["masked"] if case["masked"] else None
        state["dweights"] = 0.01 * randn(T, k)
    elif op == "permute":
        T, H, E, k = case["tokens"], case["hidden"], case["experts"], case["topk"]
        dtype = DTYPES[case["dtype"]]
        # Zipf(1.1) popularity, k different experts for each token
        popularity = -1.1 * torch.log(torch.arange(1, E + 1, device="cuda").float())[torch.argsort(rand(E))]
        gumbel = -torch.log(-torch.log(rand(T, E).clamp_(1e-20, 1 - 1e-6)))
        ids = torch.topk(popularity + gumbel, k, dim=1).indices.to(torch.int32)
        ids[rand(T) < case["dropped"]] = -1
        w = rand(T, k) + 0.05
        state["ids"], state["weights"] = ids, w / w.sum(1, keepdim=True)
        if case["backward"]:
            state["rows"] = _plan(ids, E)[1]
            state["dout"] = (0.01 * randn(T, H)).to(dtype)
            state["da"] = torch.empty(T * k, H, dtype=dtype, device="cuda").normal_(std=0.01, generator=gen)
        else:
            state["x"] = randn(T, H).to(dtype)
        state["y"] = torch.empty(T * k, H, dtype=dtype, device="cuda").normal_(generator=gen)
    elif op == "norm":
        M, C = case["rows"], case["cols"]
        dtype, wdtype = DTYPES[case["dtype"]], DTYPES[case["wdtype"]]
        # rows of different sizes and means, as the residual stream has them
        state["x"] = (randn(M, C) * (0.5 + 3 * rand(M, 1)) + randn(M, 1)).to(dtype)
        state["weight"] = (1 + 0.1 * randn(C)).to(wdtype)
        state["shift"] = (0.1 * randn(C)).to(wdtype)
        if case["backward"]:
            state["dy"] = (0.01 * randn(M, C)).to(dtype)
    else:
        for d, (n, spans) in _places(case).items():
            flat = torch.empty(n, dtype=DTYPES[d], device="cuda").normal_(std=1e-3, generator=gen)
            state["out_" + d] = torch.zeros(n, dtype=DTYPES[d], device="cuda")
            state["in_" + d] = [flat[a:a + m] for a, m in spans]
            state["to_" + d] = [state["out_" + d][a:a + m] for a, m in spans]
        state["grads"] = state["in_bf16"] + state["in_f32"]
        state["clipped"] = state["to_bf16"] + state["to_f32"]
    return state


# ---- one pass ---------------------------------------------------------------------------------------

def run(state):
    return {"route": _route, "permute": _permute, "norm": _norm, "clip": _clip}[state["op"]](state)


def _route(s):
    if own:
        from mxfp8_microscaled_precision_gb300 import mxq
        ids, w = mxq.route(s["logits"], s["topk"], score=s["score"], bias=s["bias"], n_group=s["groups"],
                           topk_group=s["kept_groups"], group_score=s["group_score"], renorm=True, scale=s["scale"],
                           token_mask=s["mask"])
        if not s["backward"]:
            return {"ids": ids, "weights": w}
        dx = mxq.route_backward(s["dweights"], s["logits"], ids, score=s["score"], renorm=True, scale=s["scale"])
        return {"ids": ids, "weights": w, "dlogits": dx}
    x = s["logits"].float() + 0.0
    T, E = x.shape
    if s["score"] == "softmax":
        e = torch.exp(x - x.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
    c = x if s["bias"] is None else p + s["bias"]
    if s["mask"] is not None:
        c = c.masked_fill(~s["mask"][:, None], -math.inf)
    if s["groups"] > 1:
        if s["group_score"] == "max":
            of_group = c.view(T, s["groups"], -1).amax(2)
        else:
            g = c if s["bias"] is not None else p.masked_fill(c == -math.inf, -math.inf)
            g = torch.sort(g.view(T, s["groups"], -1), dim=2, descending=True).values
            second = g[:, :, 1] if g.shape[2] > 1 else torch.zeros_like(g[:, :, 0])
            of_group = g[:, :, 0] + second.masked_fill(second == -math.inf, 0.0)
        best = torch.sort(of_group, dim=1, descending=True, stable=True).indices[:, :s["kept_groups"]]
        stays = torch.zeros(T, s["groups"], dtype=torch.bool, device=x.device).scatter_(1, best, True)
        c = c.masked_fill(~stays.repeat_interleave(E // s["groups"], dim=1), -math.inf)
    value, at = torch.sort(c, dim=1, descending=True, stable=True)
    value, at = value[:, :s["topk"]], at[:, :s["topk"]]
    out = value == -math.inf
    chosen = p.gather(1, at).masked_fill(out, 0.0)
    total = chosen.sum(1, keepdim=True) + RENORM_EPS
    w = s["scale"] * chosen / total
    ids = at.masked_fill(out, -1).to(torch.int32)
    if not s["backward"]:
        return {"ids": ids, "weights": w}
    dw = s["dweights"].masked_fill(out, 0.0)
    dp = ((s["scale"] * dw - (dw * w).sum(1, keepdim=True)) / total).masked_fill(out, 0.0)
    if s["score"] == "softmax":
        dx = p * (torch.zeros_like(p).scatter_(1, at, dp) - (dp * chosen).sum(1, keepdim=True))
    else:
        dx = torch.zeros_like(p).scatter_(1, at, dp * chosen * (1.0 - chosen))
    return {"ids": ids, "weights": w, "dlogits": dx.to(s["logits"].dtype)}


def _plan(ids, experts):
    """Offsets [E+1] and the row of every slot in expert order, tokens in order within an expert; a dropped
    slot's row lies behind all experts' and is given as -1 - row."""
    key = ids.reshape(-1).long()
    key = torch.where(key < 0, experts, key)
    order = torch.sort(key, stable=True).indices
    row = torch.empty_like(order).scatter_(0, order, torch.arange(key.numel(), device=key.device))
    count = torch.zeros(experts + 1, dtype=torch.int64, device=key.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.cumsum(count, 0) - count
    rows = torch.where(key < experts, row, -1 - row).to(torch.int32).view(ids.shape)
    return offsets, rows


def _permute(s):
    if own:
        from mxfp8_microscaled_precision_gb300 import mxq
        if s["backward"]:
            dy, dw = mxq.moe_combine_backward(s["dout"], s["y"], s["rows"], s["weights"])
            return {"dy": dy, "dweights": dw, "dx": mxq.moe_combine(s["da"], s["rows"])}
        offsets, rows = mxq.moe_plan(s["ids"], s["experts"])
        a = mxq.moe_dispatch(s["x"], rows)
        return {"offsets": offsets, "rows": rows, "a": a, "out": mxq.moe_combine(s["y"], rows, s["weights"])}
    if not s["backward"]:
        offsets, rows = _plan(s["ids"], s["experts"])
    else:
        rows = s["rows"]
    T, k = rows.shape
    kept = (rows >= 0)[:, :, None]
    at = torch.where(rows < 0, -1 - rows, rows).long()
    y = s["y"].float()[at].masked_fill(~kept, 0.0)
    if not s["backward"]:
        x = s["x"].float()[:, None, :].masked_fill(~kept, 0.0)
        a = torch.empty_like(s["y"])
        a[at] = x.to(a.dtype)
        out = (y * s["weights"][:, :, None]).sum(1).to(a.dtype)
        return {"offsets": offsets, "rows": rows, "a": a, "out": out}
    dout = s["dout"].float()[:, None, :]
    dy = torch.empty_like(s["y"])
    dy[at] = (s["weights"][:, :, None] * dout).masked_fill(~kept, 0.0).to(dy.dtype)
    dw = (dout * y).sum(2)
    dx = s["da"].float()[at].masked_fill(~kept, 0.0).sum(1).to(dy.dtype)
    return {"dy": dy, "dweights": dw, "dx": dx}


def _norm(s):
    if own:
        from mxfp8_microscaled_precision_gb300 import mxq
        y, mean, rstd = mxq.layer_norm(s["x"], s["weight"], s["shift"], eps=NORM_EPS)
        if not s["backward"]:
            return {"y": y, "mean": mean, "rstd": rstd}
        dx, dweight, dshift = mxq.layer_norm_backward(s["dy"], s["x"], s["weight"], mean, rstd)
        return {"y": y, "mean": mean, "rstd": rstd, "dx": dx, "dweight": dweight, "dshift": dshift}
    x, w = s["x"].float(), s["weight"].float()
    mean = x.mean(1, keepdim=True)
    rstd = 1.0 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + NORM_EPS)
    h = (x - mean) * rstd
    out = {"y": (h * w + s["shift"].float()).to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if s["backward"]:
        dy = s["dy"].float()
        u = dy * w
        dx = rstd * (u - u.mean(1, keepdim=True) - h * (u * h).mean(1, keepdim=True))
        out.update(dx=dx.to(s["x"].dtype), dweight=(dy * h).sum(0), dshift=dy.sum(0))
    return out


def _clip(s):
    if own:
        from mxfp8_microscaled_precision_gb300 import mxq
        norm, _ = mxq.clip_grad_norm(s["grads"], s["max_norm"], out=s["clipped"])
    else:
        norm = torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt()
        scale = (s["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
        [o.copy_(g.float() * scale) for o, g in zip(s["clipped"], s["grads"])]
    return {"norm": norm, "bf16": s["out_bf16"], "f32": s["out_f32"]}


# ---- what a pass has to move and compute ---------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "route":
        T, E, k, b = case["tokens"], case["experts"], case["topk"], SIZE[case["dtype"]]
        size, flops = T * E * b + 8 * T * k, 6 * T * E
        if case["backward"]:  # the logits are read by both passes, but they are one input
            size, flops = size + T * E * b + 4 * T * k, 12 * T * E
        return {"bytes": size, "flops": flops}
    if op == "permute":
        T, H, k, b = case["tokens"], case["hidden"], case["topk"], SIZE[case["dtype"]]
        wide = T * k * H * b
        if case["backward"]:  # y and da read, dy written; dout read, dx written
            return {"bytes": 3 * wide + 2 * T * H * b + 12 * T * k, "flops": 4 * T * k * H}
        return {"bytes": 2 * wide + 2 * T * H * b + 12 * T * k, "flops": 2 * T * k * H}
    if op == "norm":
        n, b = case["rows"] * case["cols"], SIZE[case["dtype"]]
        if case["backward"]:  # x and dy read, y and dx written
            return {"bytes": 4 * n * b + 8 * case["rows"] + 16 * case["cols"], "flops": 18 * n}
        return {"bytes": 2 * n * b + 8 * case["rows"] + 8 * case["cols"], "flops": 7 * n}
    sizes = _clip_sizes(case)
    return {"bytes": sum(2 * n * SIZE[d] for n, d in sizes), "flops": sum(3 * n for n, _ in sizes)}


# ---- the definitions in 64 bits ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "permute": _exact_permute, "norm": _exact_norm, "clip": _exact_clip}[case["op"]](s)


def _exact_route(s):
    x = s["logits"].double()
    T, E = x.shape
    k, n = s["topk"], s["groups"]
    p = torch.softmax(x, 1) if s["score"] == "softmax" else torch.sigmoid(x)
    c = p + s["bias"].double() if s["bias"] is not None else x
    if n > 1:
        per = E // n
        if s["group_score"] == "max":
            group = torch.stack([c[:, g * per:(g + 1) * per].max(1).values for g in range(n)], 1)
        else:
            b = c if s["bias"] is not None else p
            group = torch.stack([b[:, g * per:(g + 1) * per].topk(min(2, per), 1).values.sum(1) for g in range(n)], 1)
        # how many groups stand before this one: a higher score, or the same and a lower number
        number = torch.arange(n, device=x.device)
        before = (group[:, None, :] > group[:, :, None]) | ((group[:, None, :] == group[:, :, None]) & (number[None, :] < number[:, None]))
        gone = before.sum(2) >= s["kept_groups"]
        c = torch.where(gone[:, torch.arange(E, device=x.device) // per], -math.inf, c)
    w, at = torch.zeros(T, k, dtype=torch.float64, device=x.device), []
    for j in range(k):
        best = torch.where(c == c.max(1, keepdim=True).values, torch.arange(E, device=x.device), E).min(1).values
        at.append(best)
        w[:, j] = p[torch.arange(T, device=x.device), best]
        c = c.index_put((torch.arange(T, device=x.device), best), torch.tensor(-math.inf, dtype=torch.float64, device=x.device))
    live = s["mask"] if s["mask"] is not None else torch.ones(T, dtype=torch.bool, device=x.device)
    total = w.sum(1, keepdim=True)
    out = {"ids": None, "weights": s["scale"] * w / total * live[:, None]}
    if s["backward"]:
        # the Jacobian of w by the scores, then of the scores by the logits
        dw = s["dweights"].double()
        J = s["scale"] * (torch.eye(k, dtype=torch.float64, device=x.device) / total[:, :, None] - w[:, :, None] / total[:, :, None] ** 2)
        dp = torch.zeros_like(p).scatter_(1, torch.stack(at, 1), torch.einsum("ti,tij->tj", dw, J))
        dx = p * (dp - (p * dp).sum(1, keepdim=True)) if s["score"] == "softmax" else dp * p * torch.sigmoid(-x)
        out["dlogits"] = dx * live[:, None]
    return out


def _exact_permute(s):
    ids, (T, k) = s["ids"].long(), s["ids"].shape
    order = torch.argsort(torch.where(ids < 0, s["experts"], ids).reshape(-1), stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(T * k, device=order.device)
    place = place.view(T, k)
    H = s["y"].shape[1]
    keep = (ids >= 0).double()
    if not s["backward"]:
        a = torch.empty(T * k, H, dtype=torch.float64, device=order.device)
        out = torch.zeros(T, H, dtype=torch.float64, device=order.device)
        for j in range(k):
            a[place[:, j]] = s["x"].double() * keep[:, j, None]
            out += s["y"][place[:, j]].double() * (keep[:, j] * s["weights"][:, j].double())[:, None]
        return {"offsets": None, "rows": None, "a": a, "out": out}
    dout = s["dout"].double()
    dy = torch.empty(T * k, H, dtype=torch.float64, device=order.device)
    dw = torch.zeros(T, k, dtype=torch.float64, device=order.device)
    dx = torch.zeros(T, H, dtype=torch.float64, device=order.device)
    for j in range(k):
        dy[place[:, j]] = dout * (s["weights"][:, j].double() * keep[:, j])[:, None]
        dw[:, j] = torch.einsum("th,th->t", dout, s["y"][place[:, j]].double()) * keep[:, j]
        dx += s["da"][place[:, j]].double() * keep[:, j, None]
    return {"dy": dy, "dweights": dw, "dx": dx}


def _exact_norm(s):
    x, w, b = s["x"].double(), s["weight"].double(), s["shift"].double()
    mean = x.sum(1) / x.shape[1]
    var = torch.einsum("rc,rc->r", x - mean[:, None], x - mean[:, None]) / x.shape[1]
    rstd = (var + NORM_EPS) ** -0.5
    h = (x - mean[:, None]) * rstd[:, None]
    out = {"y": torch.addcmul(b, h, w), "mean": mean, "rstd": rstd}
    if s["backward"]:
        dy = s["dy"].double()
        dh = dy * w
        m1, m2 = dh.sum(1) / x.shape[1], torch.einsum("rc,rc->r", dh, h) / x.shape[1]
        out.update(dx=(dh - m1[:, None] - h * m2[:, None]) * rstd[:, None], dweight=torch.einsum("rc,rc->c", dy, h),
                   dshift=dy.sum(0))
    return out


def _exact_clip(s):
    total = sum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in s["grads"])
    norm = math.sqrt(total)
    scale = min(1.0, s["max_norm"] / (norm + CLIP_EPS))
    out = {"norm": torch.tensor(norm, dtype=torch.float64)}
    for d in ("bf16", "f32"):
        flat = torch.zeros(s["out_" + d].numel(), dtype=torch.float64, device="cuda")
        for g, to in zip(s["in_" + d], s["to_" + d]):
            flat[to.storage_offset():to.storage_offset() + g.numel()] = g.double() * scale
        out[d] = flat
    return out
