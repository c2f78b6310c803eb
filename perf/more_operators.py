"""Cases that measure what stands around the packed products of a layer.

Four operators, each reached as a user of packed_qmatmul_gb300 reaches it:

* experts_select: a router's logits to each token's experts and their weights
  (softmax or sigmoid scores, a bias for balance, groups, top-k, renormalised).
* apply_fused: a product of a packed weight with bias, activation (or a gate over
  pairs of rows) and residual in its epilogue.
* apply_experts_fused: the experts' products with each expert's bias and the same
  activations.
* experts_combine: the weighted sum of a token's experts, and the residual.

run() computes them either in their plain form (elementary torch operations in
32 bits, the scores that choose in 64, rounded once at the end) or, where `own` is
true, by the library's calls. exact() computes them from their definitions in 64
bits, expert by expert and choice by choice.
"""
import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decode step's token in a small model of experts
        dict(name="select_one", op="select", tokens=1, experts=32, topk=4, score="softmax", groups=1, topk_groups=1, group_score="max", bias=False,
             renormalize=True, scale=1.0, padded=0, dtype="bfloat16"),
        # a ragged batch; groups by their best expert, the last experts only pad the router's product
        dict(name="select_groups", op="select", tokens=777, experts=160, topk=6, score="softmax", groups=8, topk_groups=3, group_score="max", bias=False,
             renormalize=False, scale=16.0, padded=3, dtype="float32"),
        # a long prompt; sigmoid scores with a bias for balance, groups by their two best
        dict(name="select_prompt", op="select", tokens=16384, experts=256, topk=8, score="sigmoid", groups=8, topk_groups=4, group_score="top2", bias=True,
             renormalize=True, scale=2.5, padded=0, dtype="float32"),
        # a decode step's output projection added to the hidden state
        dict(name="fused_one", op="fused", tokens=1, n=1024, k=2048, fmt="affine", bits=4, group=64, act="none", gated=False, bias="none", residual=True),
        # a few drafted tokens through an odd layer with bias and gelu
        dict(name="fused_draft", op="fused", tokens=5, n=5001, k=1600, fmt="affine", bits=4, group=32, act="gelu", gated=False, bias="float32", residual=False),
        # a decode step's gate and up rows in turn, one large weight
        dict(name="fused_gate", op="fused", tokens=1, n=14336, k=4096, fmt="q8_0", bits=8, group=32, act="silu", gated=True, bias="none", residual=False),
        # a prompt's down projection with bias and residual
        dict(name="fused_prompt", op="fused", tokens=2048, n=4096, k=14336, fmt="q8_0", bits=8, group=32, act="none", gated=False, bias="bfloat16", residual=True),
        # decode steps of a small batch through experts with clamped gates
        dict(name="experts_decode", op="experts", tokens=16, topk=4, experts=32, n=5760, k=2880, fmt="mxfp4", bits=4, group=32, act="silu", gated=True,
             bias="bfloat16", alpha=1.702, limit=7.0, up_offset=1.0, rows="tokens"),
        # a prompt through the same experts
        dict(name="experts_prompt", op="experts", tokens=4096, topk=4, experts=32, n=5760, k=2880, fmt="mxfp4", bits=4, group=32, act="silu", gated=True,
             bias="bfloat16", alpha=1.702, limit=7.0, up_offset=1.0, rows="tokens"),
        # a shorter prompt's way back down
        dict(name="experts_down", op="experts", tokens=1000, topk=4, experts=32, n=2880, k=2880, fmt="mxfp4", bits=4, group=32, act="none", gated=False,
             bias="bfloat16", alpha=1.0, limit=0.0, up_offset=0.0, rows="positions"),
        # a decode step's sum over a token's experts
        dict(name="combine_one", op="combine", tokens=1, topk=4, n=2880, dtype="bfloat16", residual=True),
        # a prompt's
        dict(name="combine_prompt", op="combine", tokens=4096, topk=8, n=2880, dtype="bfloat16", residual=True),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    kind = rng.choice(("select", "select", "fused", "fused", "fused", "experts", "experts", "combine"))
    if kind == "select":
        groups = rng.choice((1, 1, 4, 8))
        experts = groups * _between(rng, 8, 512 // groups) if groups > 1 else _between(rng, 8, 512)
        topk_groups = rng.randint(1, groups)
        topk = min(rng.choice((1, 2, 4, 6, 8, 10)), topk_groups * (experts // groups))
        score = rng.choice(("softmax", "sigmoid"))
        bias = score == "sigmoid" and rng.random() < 0.7
        return dict(op="select", tokens=_between(rng, 1, 16384 * 256 // max(experts, 256)), experts=experts, topk=topk, score=score, groups=groups,
                    topk_groups=topk_groups, group_score=rng.choice(("max", "top2")) if groups > 1 else "max", bias=bias, renormalize=rng.random() < 0.7,
                    scale=rng.choice((1.0, 2.5)), padded=rng.choice((0, 0, 1, 5)), dtype=rng.choice(("float32", "float32", "bfloat16", "float16")))
    if kind == "combine":
        return dict(op="combine", tokens=_between(rng, 1, 4096), topk=rng.choice((1, 2, 4, 6, 8)), n=_between(rng, 200, 2880), dtype="bfloat16",
                    residual=rng.choice((True, False)))
    # Gates of more than 16 tokens on MXFP4 only: its values are exact in the tensor cores' type, the other formats' are rounded once on their way there.
    tokens = rng.choice((1, rng.randint(2, 8), rng.randint(9, 16), _between(rng, 17, 2048)))
    act, gated = rng.choice((("none", False), ("none", False), ("relu", False), ("silu", False), ("gelu", False), ("gelu_tanh", False), ("silu", True),
                             ("gelu_tanh", True)))
    fmt, bits, group = rng.choice((("affine", 4, 32), ("affine", 4, 64), ("affine", 4, 128), ("affine", 8, 64), ("q8_0", 8, 32), ("mxfp4", 4, 32),
                                   ("mxfp4_blocks", 4, 32)))
    if kind == "experts" or (gated and tokens > 16):
        fmt, bits, group = "mxfp4", 4, 32
    step = {"q8_0": 512, "mxfp4_blocks": 512}.get(fmt, group)
    k = step * max(1, round(_between(rng, 512, 4096) / step))
    n = _between(rng, 200, 14336) // 2 * 2 if gated else _between(rng, 200, 14336)
    bias = rng.choice(("none", "bfloat16", "float16", "float32"))
    if kind == "fused":
        return dict(op="fused", tokens=tokens, n=n, k=k, fmt=fmt, bits=bits, group=group, act=act, gated=gated, bias=bias, residual=rng.choice((True, False)))
    experts = rng.choice((8, 32, 64, 128))
    topk = rng.choice((1, 2, 4, 8))
    n = min(n, 5760, 5760 * 32 // experts)
    n -= n % 16  # whole matrices of scales on 16-byte boundaries, as checkpoints lay them out
    clamped = act == "silu" and gated and rng.random() < 0.5
    return dict(op="experts", tokens=_between(rng, 1, 16384 // topk), topk=topk, experts=experts, n=max(n, 16), k=min(k, 2880), fmt=fmt, bits=bits,
                group=group, act=act, gated=gated, bias=bias, alpha=1.702 if clamped else 1.0, limit=7.0 if clamped else 0.0, up_offset=1.0 if clamped else 0.0,
                rows=rng.choice(("tokens", "positions")))


# ---------------------------------------------------------------- inputs
def _normal(gen, shape, dtype, sigma=1.0, mean=0.0):
    return (torch.randn(shape, generator=gen, device=DEVICE) * sigma + mean).to(dtype)


def _bytes(gen, shape, lo=0, hi=256):
    return torch.randint(lo, hi, shape, generator=gen, device=DEVICE, dtype=torch.uint8)


def _weight(case, gen, lead):
    """Packed parts of a weight [*lead, n, k], its values about 1 / sqrt(k) in size."""
    n, k, fmt = case["n"], case["k"], case["fmt"]
    size, rows = k ** -0.5, (*lead, n)
    s = {}
    if fmt == "affine":
        codes = 1 << case["bits"]
        s["codes"] = _bytes(gen, (*rows, k * case["bits"] // 8))
        scale = (torch.rand((*rows, k // case["group"]), generator=gen, device=DEVICE) + 0.5) * size * 3.5 / codes
        s["scales"] = scale.to(torch.bfloat16)
        s["biases"] = (scale * codes * -0.5 * _normal(gen, scale.shape, torch.float32, 0.05, 1.0)).to(torch.bfloat16)
    elif fmt == "q8_0":
        blocks = torch.empty((*rows, k // 32, 34), dtype=torch.uint8, device=DEVICE)
        d = (torch.rand((*rows, k // 32), generator=gen, device=DEVICE) + 0.5) * size / 73
        blocks[..., :2] = d.half().unsqueeze(-1).view(torch.uint8)
        blocks[..., 2:] = torch.randint(-127, 128, (*rows, k // 32, 32), generator=gen, device=DEVICE, dtype=torch.int8).view(torch.uint8)
        s["codes"] = blocks.flatten(-2)
    else:
        low = 127 + round(math.log2(size)) - 2
        if fmt == "mxfp4":
            s["codes"] = _bytes(gen, (*rows, k // 2))
            s["scales"] = _bytes(gen, (*rows, k // 32), low, low + 3)
        else:
            blocks = _bytes(gen, (*rows, k // 32, 17))
            blocks[..., 0] = _bytes(gen, (*rows, k // 32), low, low + 3)
            s["codes"] = blocks.flatten(-2)
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    T = case["tokens"]
    s = dict(case=case)
    if case["op"] == "select":
        E = case["experts"]
        logits = _normal(gen, (T, E), DTYPES[case["dtype"]], 1.5)
        if case["padded"]:
            logits[:, E - case["padded"]:] = -math.inf
        s["logits"] = logits
        s["bias"] = _normal(gen, (E,), torch.float32, 0.05) if case["bias"] else None
        if own:
            import packed_qmatmul_gb300 as qm

            s["router"] = qm.Router(case["topk"], score=case["score"], bias=s["bias"], groups=case["groups"], topk_groups=case["topk_groups"],
                                    group_score=case["group_score"], renormalize=case["renormalize"], scale=case["scale"])
        return s
    if case["op"] == "combine":
        s["y"] = _normal(gen, (T, case["topk"], case["n"]), DTYPES[case["dtype"]])
        weights = torch.rand((T, case["topk"]), generator=gen, device=DEVICE) + 0.05
        s["weights"] = weights / weights.sum(-1, keepdim=True)
        s["residual"] = _normal(gen, (T, case["n"]), DTYPES[case["dtype"]]) if case["residual"] else None
        return s
    n, k = case["n"], case["k"]
    experts = case["op"] == "experts"
    lead = (case["experts"],) if experts else ()
    s |= _weight(case, gen, lead)
    s["bias"] = None if case["bias"] == "none" else _normal(gen, (*lead, n), DTYPES[case["bias"]], 0.5)
    if experts:
        P = T * case["topk"]
        s["ids"] = torch.rand((T, case["experts"]), generator=gen, device=DEVICE).argsort(1)[:, : case["topk"]].to(torch.int32).contiguous()
        s["x"] = _normal(gen, (T if case["rows"] == "tokens" else P, k), torch.bfloat16)
        s["most"] = int(torch.bincount(s["ids"].flatten(), minlength=1).max())  # positions of the busiest expert
    else:
        s["x"] = _normal(gen, (T, k), torch.bfloat16)
        s["residual"] = _normal(gen, (T, n // 2 if case["gated"] else n), torch.bfloat16) if case["residual"] else None
    if own:
        import packed_qmatmul_gb300 as qm

        s["w"] = qm.QWeight(case["fmt"], (*lead, n, k), s["codes"], s.get("scales"), s.get("biases"), bits=case["bits"],
                            group_size=case["group"], flags=qm.QM_WEIGHT_STATIC)
        s["epilogue"] = qm.Epilogue(bias=s["bias"], act=case["act"], gated=case["gated"], alpha=case.get("alpha", 1.0), limit=case.get("limit", 0.0),
                                    up_offset=case.get("up_offset", 0.0))
        if experts:
            s["workspace"] = torch.empty(max(256, qm.qm_apply_experts_workspace(s["w"], T, case["topk"])), dtype=torch.uint8, device=DEVICE)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if own:
        import packed_qmatmul_gb300 as qm

        if case["op"] == "select":
            ids, weights = qm.experts_select(s["logits"], s["router"])
            return {"ids": ids, "weights": weights}
        if case["op"] == "combine":
            return {"out": qm.experts_combine(s["y"], s["weights"], s["residual"])}
        if case["op"] == "experts":
            return {"y": qm.apply_experts_fused(s["w"], s["ids"], s["x"], s["epilogue"], workspace=s["workspace"])}
        return {"y": qm.apply_fused(s["w"], s["x"], s["epilogue"], s["residual"])}
    if case["op"] == "select":
        return _plain_select(s)
    if case["op"] == "combine":
        out = (s["y"].float() * s["weights"][..., None]).sum(1)
        return {"out": (out if s["residual"] is None else out + s["residual"].float()).to(s["y"].dtype)}
    value = _plain_values(s)
    if case["op"] == "fused":
        v = s["x"].float() @ value.T
        if s["bias"] is not None:
            v = v + s["bias"].float()
        v = _plain_act(case, v)
        return {"y": (v if s["residual"] is None else v + s["residual"].float()).to(torch.bfloat16)}
    # Each expert's positions side by side, as many places to an expert as the busiest needs.
    E, n, k = value.shape
    ids = s["ids"].flatten().long()
    order = ids.argsort(stable=True)
    expert = ids[order]
    starts = torch.searchsorted(expert, torch.arange(E, device=DEVICE))
    place = torch.arange(ids.numel(), device=DEVICE) - starts[expert]
    row = order // case["topk"] if case["rows"] == "tokens" else order
    x = torch.zeros((E, s["most"], k), device=DEVICE)
    x[expert, place] = s["x"][row].float()
    v = torch.bmm(x, value.transpose(1, 2))[expert, place]
    if s["bias"] is not None:
        v = v + s["bias"].float()[expert]
    v = _plain_act(case, v).to(torch.bfloat16)
    y = torch.empty_like(v)
    y[order] = v
    return {"y": y.view(case["tokens"], case["topk"], -1)}


def _plain_act(case, v):
    """The activation of v, or of its gates (even columns) times the columns beside them, in 32 bits."""
    g = v[..., 0::2] if case["gated"] else v
    limit, alpha = case.get("limit", 0.0), case.get("alpha", 1.0)
    if limit:
        g = g.clamp(max=limit)
    if case["act"] == "relu":
        a = g.clamp(min=0.0)
    elif case["act"] == "silu":
        a = g / (1.0 + (g * -alpha).exp())
    elif case["act"] == "gelu":
        a = g * 0.5 * torch.erfc(g * -(0.5 ** 0.5))
    elif case["act"] == "gelu_tanh":
        a = g / (1.0 + ((g + 0.044715 * g * g * g) * (-2.0 * (2.0 / math.pi) ** 0.5)).exp())
    else:
        a = g
    if not case["gated"]:
        return a
    u = v[..., 1::2]
    if limit:
        u = u.clamp(-limit, limit)
    return a * (u + case.get("up_offset", 0.0))


def _plain_values(s):
    """The packed weight's values in 32 bits."""
    case = s["case"]
    if case["fmt"] == "affine":
        c = s["codes"]
        if case["bits"] == 4:
            c = torch.stack([c & 15, c >> 4], -1).flatten(-2)
        c = c.float().unflatten(-1, (-1, case["group"]))
        return (c * s["scales"].float()[..., None] + s["biases"].float()[..., None]).flatten(-2)
    if case["fmt"] == "q8_0":
        b = s["codes"].unflatten(-1, (-1, 34))
        return (b[..., 2:].contiguous().view(torch.int8).float() * b[..., :2].contiguous().view(torch.float16).float()).flatten(-2)
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEVICE)
    if case["fmt"] == "mxfp4":
        c, scale = s["codes"].unflatten(-1, (-1, 16)), s["scales"]
        c = torch.stack([c & 15, c >> 4], -1).flatten(-2)
    else:
        b = s["codes"].unflatten(-1, (-1, 17))
        c, scale = b[..., 1:], b[..., 0]
        c = torch.cat([c & 15, c >> 4], -1)
    return (table[c.int()] * (scale.float() - 127.0).exp2()[..., None]).flatten(-2)


def _plain_select(s):
    """Choices by scores in 64 bits (values next to a border), weights in 32."""
    case, topk = s["case"], s["case"]["topk"]
    T, E = s["logits"].shape
    wide = s["logits"].double()
    score = torch.softmax(wide, -1) if case["score"] == "softmax" else torch.sigmoid(wide)
    key = score if s["bias"] is None else score + s["bias"].double()
    key = key.masked_fill(wide == -math.inf, -math.inf)
    if case["groups"] > 1:
        grouped = key.view(T, case["groups"], -1)
        best = grouped.sort(dim=-1, descending=True).values[..., : 2 if case["group_score"] == "top2" else 1].sum(-1)
        kept = best.sort(dim=-1, descending=True, stable=True).indices[:, : case["topk_groups"]]
        stays = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True)
        key = grouped.masked_fill(~stays[..., None], -math.inf).view(T, E)
    top = key.sort(dim=-1, descending=True, stable=True)
    ids = top.indices[:, :topk]
    found = top.values[:, :topk] > -math.inf
    logits = s["logits"].float()
    if case["score"] == "softmax":
        weights = torch.softmax(logits, -1).gather(1, ids)
    else:
        weights = torch.sigmoid(logits).gather(1, ids)
    weights = weights.masked_fill(~found, 0.0)
    if case["renormalize"]:
        weights = weights / weights.sum(-1, keepdim=True)
    return {"ids": ids.masked_fill(~found, -1).to(torch.int32), "weights": weights * case["scale"]}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    T = case["tokens"]
    if case["op"] == "select":
        E, topk = case["experts"], case["topk"]
        return {"bytes": T * (E * (4 if case["dtype"] == "float32" else 2) + topk * 8) + E * 4 * case["bias"], "flops": T * E * 6}
    if case["op"] == "combine":
        rows = case["topk"] + 1 + case["residual"]
        return {"bytes": T * (rows * case["n"] * 2 + case["topk"] * 4), "flops": T * case["n"] * (2 * case["topk"] + case["residual"])}
    n, k = case["n"], case["k"]
    out = n // 2 if case["gated"] else n
    row = {"affine": k * case["bits"] // 8 + k // case["group"] * 4, "q8_0": k // 32 * 34, "mxfp4": k // 32 * 17, "mxfp4_blocks": k // 32 * 17}[case["fmt"]]
    row += {"none": 0, "float32": 4}.get(case["bias"], 2)
    if case["op"] == "fused":
        return {"bytes": n * row + T * (k * 2 + out * 2 * (1 + case["residual"])), "flops": 2 * T * n * k}
    # The experts that some token goes to, in the mean over even choices.
    E, topk = case["experts"], case["topk"]
    used = E * (1.0 - (1.0 - topk / E) ** T)
    x_rows = T if case["rows"] == "tokens" else T * topk
    return {"bytes": used * n * row + x_rows * k * 2 + T * topk * (out * 2 + 4), "flops": 2 * T * topk * n * k}


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_rows(case, codes, scales, biases):
    """The values of packed rows [n, ...] in 64 bits, a block's parts taken one by one."""
    n, k = codes.shape[0], case["k"]
    w = torch.empty((n, k), dtype=torch.float64, device=DEVICE)
    if case["fmt"] == "affine":
        per = 8 // case["bits"]
        scale, low = scales.double().repeat_interleave(case["group"], 1), biases.double().repeat_interleave(case["group"], 1)
        for i in range(per):
            w[:, i::per] = ((codes.int() >> (i * case["bits"])) % (1 << case["bits"])).double()
        return w * scale + low
    if case["fmt"] == "q8_0":
        for i in range(k // 32):
            block = codes[:, 34 * i: 34 * i + 34].contiguous()
            w[:, 32 * i: 32 * i + 32] = block[:, 2:].contiguous().view(torch.int8).double() * block[:, :2].contiguous().view(torch.float16).double()
        return w

    def value(c):  # sign, two bits of exponent, one of mantissa
        e, m = (c // 2) % 4, (c % 2).double()
        return torch.where(e == 0, m / 2, (1 + m / 2) * torch.pow(2.0, e.double() - 1)) * (1 - 2 * (c // 8).double())

    for i in range(k // 32):
        if case["fmt"] == "mxfp4":
            block, s = codes[:, 16 * i: 16 * i + 16].int(), scales[:, i].double()
            lo, hi = w[:, 32 * i: 32 * i + 32: 2], w[:, 32 * i + 1: 32 * i + 32: 2]
        else:
            block, s = codes[:, 17 * i + 1: 17 * i + 17].int(), codes[:, 17 * i].double()
            lo, hi = w[:, 32 * i: 32 * i + 16], w[:, 32 * i + 16: 32 * i + 32]
        s = torch.pow(2.0, s - 127.0)[:, None]
        lo.copy_(value(block % 16) * s)
        hi.copy_(value(block // 16) * s)
    return w


def _exact_epilogue(case, v, bias, residual=None):
    if bias is not None:
        v = v + bias.double()
    g, u = (v[:, 0::2], v[:, 1::2]) if case["gated"] else (v, None)
    limit = case.get("limit", 0.0) or math.inf
    g = torch.where(g > limit, torch.full_like(g, limit), g) if case["gated"] else g
    act = case["act"]
    if act == "relu":
        g = torch.where(g > 0, g, torch.zeros_like(g))
    elif act == "silu":
        g = g * torch.special.expit(case.get("alpha", 1.0) * g)
    elif act == "gelu":
        g = g * torch.special.ndtr(g)
    elif act == "gelu_tanh":
        g = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
    if case["gated"]:
        g = g * (torch.clamp(u, -limit, limit) + case.get("up_offset", 0.0))
    return g if residual is None else g + residual.double()


def _exact_select(s):
    case = s["case"]
    x = s["logits"].double()
    T, E = x.shape
    if case["score"] == "softmax":
        e = torch.exp(x - x.max(-1, keepdim=True).values)
        score = e / e.sum(-1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-x))
    key = torch.where(torch.isinf(x), x, score if s["bias"] is None else score + s["bias"].double())
    where = torch.arange(T, device=DEVICE)
    if case["groups"] > 1:
        size = E // case["groups"]
        best = torch.empty((T, case["groups"]), dtype=torch.float64, device=DEVICE)
        for g in range(case["groups"]):
            part = key[:, g * size: (g + 1) * size].clone()
            first, at = part.max(-1)
            best[:, g] = first
            if case["group_score"] == "top2":
                part[where, at] = -math.inf
                best[:, g] += part.max(-1).values
        open_ = torch.zeros((T, case["groups"]), dtype=torch.bool, device=DEVICE)
        rank = (best[:, None, :] > best[:, :, None]).sum(-1)  # groups strictly better
        for g in range(case["groups"]):
            ties = (best[:, :g] == best[:, g: g + 1]).sum(-1)
            open_[:, g] = rank[:, g] + ties < case["topk_groups"]
        key = torch.where(open_.repeat_interleave(size, 1), key, torch.full_like(key, -math.inf))
    ids = torch.empty((T, case["topk"]), dtype=torch.int32, device=DEVICE)
    weights = torch.empty((T, case["topk"]), dtype=torch.float64, device=DEVICE)
    place = torch.arange(E, device=DEVICE)
    for j in range(case["topk"]):
        top = key.max(-1, keepdim=True).values
        at = torch.where(key == top, place, E).min(-1).values
        got = top[:, 0] > -math.inf
        ids[:, j] = torch.where(got, at, -1).int()
        weights[:, j] = torch.where(got, score[where, at], 0.0)
        key[where, at] = -math.inf
    if case["renormalize"]:
        weights = weights / weights.sum(-1, keepdim=True)
    return {"ids": ids, "weights": weights * case["scale"]}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "select":
        return _exact_select(s)
    if case["op"] == "combine":
        out = torch.zeros((case["tokens"], case["n"]), dtype=torch.float64, device=DEVICE) if s["residual"] is None else s["residual"].double()
        for j in range(case["topk"]):
            out = out + s["weights"][:, j, None].double() * s["y"][:, j].double()
        return {"out": out}
    if case["op"] == "fused":
        w = _exact_rows(case, s["codes"], s.get("scales"), s.get("biases"))
        return {"y": _exact_epilogue(case, s["x"].double() @ w.T, s["bias"], s["residual"])}
    out = case["n"] // 2 if case["gated"] else case["n"]
    flat = s["ids"].flatten()
    y = torch.zeros((flat.numel(), out), dtype=torch.float64, device=DEVICE)
    for e in range(case["experts"]):
        at = (flat == e).nonzero()[:, 0]
        if at.numel():
            w = _exact_rows(case, s["codes"][e], s["scales"][e], None)
            x = s["x"][at // case["topk"] if case["rows"] == "tokens" else at].double()
            y[at] = _exact_epilogue(case, x @ w.T, None if s["bias"] is None else s["bias"][e])
    return {"y": y.view(case["tokens"], case["topk"], out)}
