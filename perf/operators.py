"""Cases that measure the operators around a paged key/value cache.

Three operators, each reached as a user of packed_qmatmul_gb300 reaches it:

* head_norm_rope: RMS norm of every head of the queries and keys and the
  rotation by position, in one pass over the rows of a fused q/k/v product.
* cache_append: the new tokens' keys (normed and rotated on the way) and values
  into the pages of a paged cache.
* cache_attend: attention of each sequence's new tokens (one token, a few
  drafted ones or a chunk of a prompt) over its pages, causal, optionally within
  a window; a cache of 16-bit values or of 8-bit codes with a scale per token
  and head.

run() computes them either in their plain form (elementary torch operations in
32 bits, rounded once at the end) or, where `own` is true, by the library's
calls. exact() computes them from their definitions in 64 bits, sequence by
sequence and head by head.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
DTYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16}
EPS = 1e-6
THETA = 1e6


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of one user: the query and key heads of a single token
        dict(name="norm_rope_one", op="norm_rope", tokens=1, heads=16, kv_heads=8, dim=128, rot=128, style="half", dtype="bfloat16"),
        # a ragged mix of prompts, rotated in adjacent pairs over half of each head
        dict(name="norm_rope_ragged", op="norm_rope", tokens=777, heads=20, kv_heads=4, dim=96, rot=48, style="pairs", dtype="float16"),
        # a long prompt's projections
        dict(name="norm_rope_prompt", op="norm_rope", tokens=16384, heads=16, kv_heads=8, dim=128, rot=128, style="half", dtype="bfloat16"),
        # a decode step of a batch: one new token a sequence
        dict(name="append_decode", op="append", seqs=64, new_min=1, new_max=1, len_min=1, len_max=200, idle=3, kv_heads=8, dim=128, rot=128,
             style="half", page=16, dtype="bfloat16", norm=True),
        # chunks of odd lengths over pages that are no power of two
        dict(name="append_chunks", op="append", seqs=9, new_min=1, new_max=301, len_min=301, len_max=900, idle=1, kv_heads=5, dim=80, rot=80,
             style="pairs", page=48, dtype="float16", norm=False),
        # four prompts stored at once
        dict(name="append_prompts", op="append", seqs=4, new_min=4096, new_max=4096, len_min=4096, len_max=4096, idle=0, kv_heads=8, dim=128,
             rot=128, style="half", page=64, dtype="bfloat16", norm=True),
        # one user's decode step after a short conversation
        dict(name="attend_one", op="attend", seqs=1, new_min=1, new_max=1, len_min=1500, len_max=1500, idle=0, heads=16, kv_heads=8, dim=128,
             page=16, window=0, dtype="bfloat16", codes=False, lse=False),
        # a serving batch's decode step: ragged lengths and a few empty slots
        dict(name="attend_decode", op="attend", seqs=64, new_min=1, new_max=1, len_min=1, len_max=8192, idle=2, heads=16, kv_heads=8, dim=128,
             page=16, window=0, dtype="bfloat16", codes=False, lse=False),
        # decode over long documents held as 8-bit codes
        dict(name="attend_long_codes", op="attend", seqs=4, new_min=1, new_max=1, len_min=65536, len_max=131072, idle=0, heads=32, kv_heads=8,
             dim=128, page=64, window=0, dtype="bfloat16", codes=True, lse=True),
        # drafted tokens verified together, seven query heads to a key head
        dict(name="attend_draft", op="attend", seqs=32, new_min=5, new_max=5, len_min=100, len_max=4000, idle=0, heads=14, kv_heads=2, dim=64,
             page=32, window=0, dtype="float16", codes=False, lse=False),
        # chunks of prompts beside decoding sequences, within a window
        dict(name="attend_mixed", op="attend", seqs=7, new_min=1, new_max=613, len_min=700, len_max=5000, idle=1, heads=16, kv_heads=4, dim=96,
             page=48, window=2000, dtype="float16", codes=False, lse=True),
        # one chunk of a long prompt over what is already in the cache
        dict(name="attend_prompt", op="attend", seqs=1, new_min=4096, new_max=4096, len_min=32768, len_max=32768, idle=0, heads=16, kv_heads=8,
             dim=128, page=64, window=0, dtype="bfloat16", codes=False, lse=False),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    kind = rng.choice(("norm_rope", "append", "decode", "decode", "draft", "chunk", "chunk"))
    dim = rng.choice((64, 80, 96, 128, 128))
    dtype = rng.choice(("bfloat16", "float16"))
    page = rng.choice((16, 32, 48, 64, 256))
    kv_heads = rng.choice((1, 2, 4, 5, 8))
    if kind == "norm_rope":
        return dict(op="norm_rope", tokens=_between(rng, 1, 16384), heads=kv_heads * rng.choice((1, 2, 3)), kv_heads=kv_heads, dim=dim,
                    rot=rng.choice((dim, dim, dim // 2)), style=rng.choice(("half", "pairs")), dtype=dtype)
    if kind == "append":
        new = _between(rng, 1, 4096)
        seqs = _between(rng, 1, max(1, min(64, 16384 // new)))
        return dict(op="append", seqs=seqs, new_min=rng.randint(1, new), new_max=new, len_min=new, len_max=new + rng.randint(0, 1000),
                    idle=rng.choice((0, 0, 1)) if seqs > 2 else 0, kv_heads=kv_heads, dim=dim, rot=rng.choice((dim, dim, dim // 2)),
                    style=rng.choice(("half", "pairs")), page=page, dtype=dtype, norm=rng.choice((True, False)))
    heads = kv_heads * rng.choice((1, 2, 4, 7))
    case = dict(op="attend", heads=heads, kv_heads=kv_heads, dim=dim, page=page, window=rng.choice((0, 0, 0, 513)), dtype=dtype,
                codes=rng.random() < 0.3, lse=rng.choice((True, False)))
    if kind == "chunk":
        new = _between(rng, 17, 4096)
        seqs = _between(rng, 1, max(1, 4096 // new))
        most = max(new, min(32768, int(1.5e9 / (new * seqs * heads))))
        length = _between(rng, new, most)
        case |= dict(seqs=seqs, new_min=rng.choice((new, 1)), new_max=new, len_min=max(new, length // 2), len_max=length)
    else:
        new = 1 if kind == "decode" else rng.randint(2, 8)
        length = _between(rng, 16, 65536)
        seqs = _between(rng, 1, max(1, min(64, int(4e8 / (length * kv_heads * dim)), int(1e8 / (length * heads * new)))))
        case |= dict(seqs=seqs, new_min=1, new_max=new, len_min=max(new, length // rng.choice((1, 4))), len_max=length)
    return case | dict(idle=1 if case["seqs"] > 3 and rng.random() < 0.3 else 0)


def _lengths(case):
    """[(new tokens, length with them)] of each sequence: fixed by the case's own numbers."""
    rng = random.Random("%(seqs)d %(new_min)d %(new_max)d %(len_min)d %(len_max)d %(page)d" % case)
    got = []
    for i in range(case["seqs"]):
        new = case["new_max"] if i == 0 else rng.randint(case["new_min"], case["new_max"])
        got.append((new, max(new, case["len_max"] if i == 0 else rng.randint(case["len_min"], case["len_max"]))))
    for i in range(case["idle"]):  # slots of a batch that hold no sequence: their rows attend to nothing and store nothing
        got[-1 - i] = (got[-1 - i][0], 0)
    return got


# ---------------------------------------------------------------- inputs
def _table(case, rows):
    """The rotation's cosines and sines, [rows, rot]: rot / 2 of each."""
    half = case["rot"] // 2
    at = torch.arange(rows, device=DEVICE, dtype=torch.float64)
    angle = at[:, None] * THETA ** (-torch.arange(half, device=DEVICE, dtype=torch.float64) / half)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _normal(gen, shape, dtype, sigma=1.0, mean=0.0):
    return (torch.randn(shape, generator=gen, device=DEVICE) * sigma + mean).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    dtype, dim, kv = DTYPES[case["dtype"]], case["dim"], case["kv_heads"]
    s = dict(case=case)
    if case["op"] == "norm_rope":
        # q, k and v side by side, as one product of the fused weight leaves them
        T, heads = case["tokens"], case["heads"]
        rows = _normal(gen, (T, (heads + 2 * kv) * dim), dtype, 1.7)
        s["q"] = rows[:, : heads * dim].unflatten(1, (heads, dim))
        s["k"] = rows[:, heads * dim: (heads + kv) * dim].unflatten(1, (kv, dim))
        s["q_weight"], s["k_weight"] = (_normal(gen, (dim,), dtype, 0.2, 1.0) for _ in range(2))
        most = 4 * max(T, 2048)
        s["table"] = _table(case, most)
        s["positions"] = torch.randint(0, most, (T,), generator=gen, device=DEVICE, dtype=torch.int32)
        if own:
            import packed_qmatmul_gb300 as qm

            s["rope"] = qm.Rope(s["table"], style=case["style"])
        return s
    # a paged cache: every sequence's pages lie scattered over it
    page, lens = case["page"], _lengths(case)
    need = [-(-n // page) for _, n in lens]
    width = max(need) + 1
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=gen, device=DEVICE).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    first = 0
    perm = order.cpu()
    for i, n in enumerate(need):
        table[i, :n] = perm[first: first + n]
        first += n
    s["page_table"] = table.to(DEVICE)
    s["lens"] = torch.tensor([n for _, n in lens], dtype=torch.int32, device=DEVICE)
    offsets = [0]
    for new, _ in lens:
        offsets.append(offsets[-1] + new)
    T = offsets[-1]
    s["q_offsets"] = torch.tensor(offsets, dtype=torch.int32, device=DEVICE)
    s["tokens"], s["max_new"], s["max_len"] = T, max(new for new, _ in lens), max(n for _, n in lens)
    shape = (pages, kv, page, dim)
    if case.get("codes"):
        for part in ("k", "v"):
            s[part + "_cache"] = torch.randint(-127, 128, shape, generator=gen, device=DEVICE, dtype=torch.int8)
            s[part + "_scales"] = torch.rand(shape[:-1], generator=gen, device=DEVICE) * 0.02 + 0.01
    else:
        s["k_cache"], s["v_cache"] = (_normal(gen, shape, dtype) for _ in range(2))
    if own:
        import packed_qmatmul_gb300 as qm

        s["cache"] = qm.Cache(s["k_cache"], s["v_cache"], s.get("k_scales"), s.get("v_scales"))
        s["batch"] = qm.Batch(s["lens"], s["page_table"], s["q_offsets"], tokens=T, max_new=s["max_new"])
    if case["op"] == "append":
        rows = _normal(gen, (T, 2 * kv * dim), dtype, 1.7)
        s["k"] = rows[:, : kv * dim].unflatten(1, (kv, dim))
        s["v"] = rows[:, kv * dim:].unflatten(1, (kv, dim))
        s["k_weight"] = _normal(gen, (dim,), dtype, 0.2, 1.0) if case["norm"] else None
        s["table"] = _table(case, s["max_len"])
        s["held"] = torch.tensor([t for i, (_, n) in enumerate(lens) if n for t in range(offsets[i], offsets[i + 1])], device=DEVICE)
        if own:
            s["rope"] = qm.Rope(s["table"], style=case["style"])
    else:
        s["q"] = _normal(gen, (T, case["heads"], dim), dtype, 1.7)
        s["scale"] = dim ** -0.5
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if own:
        import packed_qmatmul_gb300 as qm

        if case["op"] == "norm_rope":
            q, k = qm.head_norm_rope([s["q"], s["k"]], s["positions"], s["rope"], weights=[s["q_weight"], s["k_weight"]], eps=EPS)
            return {"q": q, "k": k}
        if case["op"] == "append":
            qm.cache_append(s["cache"], s["batch"], s["k"], s["v"], s["rope"], k_weight=s["k_weight"], eps=EPS)
            return {"k": s["k_cache"], "v": s["v_cache"]}
        out = qm.cache_attend(s["cache"], s["batch"], s["q"], scale=s["scale"], window=case["window"], lse=case["lse"])
        return {"out": out[0], "lse": out[1]} if case["lse"] else {"out": out}
    if case["op"] == "norm_rope":
        at = s["positions"].long()
        return {"q": _plain_norm_rope(s["q"], s["q_weight"], at, s), "k": _plain_norm_rope(s["k"], s["k_weight"], at, s)}
    if case["op"] == "append":
        return _plain_append(s)
    return _plain_attend(s)


def _plain_norm_rope(x, weight, at, s):
    """The head norm and the rotation of x [tokens, heads, dim] at 32 bits, rounded once."""
    rot = s["case"]["rot"]
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * weight.float()
    angle = s["table"][at][:, None]
    cos, sin = angle[..., : rot // 2], angle[..., rot // 2:]
    if s["case"]["style"] == "half":
        a, b = y[..., : rot // 2], y[..., rot // 2: rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)


def _places(s):
    """Each new token's sequence, place within its sequence's new tokens, and position (negative where its slot is idle)."""
    offsets = s["q_offsets"].long()
    token = torch.arange(s["tokens"], device=DEVICE)
    seq = torch.bucketize(token, offsets[1:], right=True)
    place = token - offsets[seq]
    return seq, place, s["lens"].long()[seq] - (offsets[seq + 1] - offsets[seq]) + place


def _plain_append(s):
    page = s["case"]["page"]
    seq, _, at = _places(s)
    k = _plain_norm_rope(s["k"], s["k_weight"], at.clamp(min=0), s)
    held = s["held"]
    seq, at = seq[held], at[held]
    slot = s["page_table"].long()[seq, at // page]
    s["k_cache"][slot, :, at % page] = k[held]
    s["v_cache"][slot, :, at % page] = s["v"][held]
    return {"k": s["k_cache"], "v": s["v_cache"]}


def _plain_attend(s):
    case = s["case"]
    heads, kv, dim = case["heads"], case["kv_heads"], case["dim"]
    seqs, group, new, most = case["seqs"], case["heads"] // case["kv_heads"], s["max_new"], s["max_len"]
    seq, place, at = _places(s)
    q = torch.zeros((seqs, new, heads, dim), device=DEVICE)
    q[seq, place] = s["q"].float()
    pos = torch.full((seqs, new), -1, device=DEVICE)
    pos[seq, place] = at
    q = q.view(seqs, new, kv, group, dim).permute(0, 2, 3, 1, 4).reshape(seqs, kv, group * new, dim)
    held = s["page_table"].long().clamp(min=0)

    def rows(part):  # every sequence's keys or values in order, [seqs, kv_heads, most, dim]
        x = s[part + "_cache"][held].float()
        if case["codes"]:
            x = x * s[part + "_scales"][held][..., None]
        return x.permute(0, 2, 1, 3, 4).flatten(2, 3)[:, :, :most]

    key = torch.arange(most, device=DEVICE)
    seen = key <= pos[..., None]
    if case["window"]:
        seen &= key > pos[..., None] - case["window"]
    score = (q * s["scale"]) @ rows("k").transpose(-1, -2)
    score = score.view(seqs, kv, group, new, most).masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = score.sub_(top).exp_().view(seqs, kv, group * new, most)
    total = p.sum(-1, keepdim=True)
    out = (p @ rows("v")) / total.clamp(min=1e-30)
    out = out.view(seqs, heads, new, dim)[seq, :, place].to(s["q"].dtype)
    if not case["lse"]:
        return {"out": out}
    lse = top + total.log().view_as(top)
    return {"out": out, "lse": lse.view(seqs, heads, new)[seq, :, place]}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    dim, kv = case["dim"], case["kv_heads"]
    if case["op"] == "norm_rope":
        heads = case["heads"] + kv
        return {"bytes": case["tokens"] * (heads * dim * 2 * 2 + case["rot"] * 4 + 4) + 2 * dim * 2,
                "flops": case["tokens"] * heads * (4 * dim + 3 * case["rot"])}
    lens = _lengths(case)
    if case["op"] == "append":
        kept = sum(new for new, n in lens if n)
        return {"bytes": kept * (2 * kv * dim * 2 * 2 + case["rot"] * 4),
                "flops": kept * kv * (4 * dim * case["norm"] + 3 * case["rot"])}
    window, heads = case["window"] or 1 << 40, case["heads"]
    one = kv * (dim + 4 if case["codes"] else 2 * dim)  # bytes of one token's keys, or values
    size = sum(new for new, _ in lens) * heads * (2 * dim * 2 + 4 * case["lse"])
    pairs = 0
    for new, n in lens:
        if n:
            size += 2 * one * (n - max(0, n - new - window + 1))
            full = max(0, min(new, n - window))  # the last `full` new tokens see a whole window, the others all before them
            pairs += full * window + sum(range(n - new + 1, n - full + 1))
    return {"bytes": size, "flops": 4 * pairs * heads * dim}


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_norm_rope(x, weight, positions, table, style, rot):
    """Token by token quantities of one head axis, x [tokens, heads, dim] in 64 bits."""
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * weight.double()
    y = x.clone()
    half = rot // 2
    t = table.double()[positions]
    for i in range(half):
        a, b = (i, i + half) if style == "half" else (2 * i, 2 * i + 1)
        c, z = t[:, i, None], t[:, half + i, None]
        y[..., a] = x[..., a] * c - x[..., b] * z
        y[..., b] = x[..., b] * c + x[..., a] * z
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        at = s["positions"].long()
        return {n: _exact_norm_rope(s[n].double(), s[n + "_weight"], at, s["table"], case["style"], case["rot"]) for n in ("q", "k")}
    page, lens = case["page"], _lengths(case)
    table = s["page_table"].cpu()
    if case["op"] == "append":
        k, v = s["k_cache"].double(), s["v_cache"].double()
        first = 0
        for i, (new, n) in enumerate(lens):
            if n:
                at = torch.arange(n - new, n)
                slot = table[i].long()[at // page].to(DEVICE)
                at = at.to(DEVICE)
                k[slot, :, at % page] = _exact_norm_rope(s["k"][first: first + new].double(), s["k_weight"], at, s["table"], case["style"], case["rot"])
                v[slot, :, at % page] = s["v"][first: first + new].double()
            first += new
        return {"k": k, "v": v}
    heads, kv, dim = case["heads"], case["kv_heads"], case["dim"]
    out = torch.zeros((s["tokens"], heads, dim), device=DEVICE, dtype=torch.float64)
    lse = torch.full((s["tokens"], heads), -math.inf, device=DEVICE, dtype=torch.float64)
    first = 0
    for i, (new, n) in enumerate(lens):
        slots = table[i, : -(-n // page)].long().to(DEVICE)
        for h in range(kv if n else 0):
            kd, vd = s["k_cache"][slots, h].double(), s["v_cache"][slots, h].double()
            if case["codes"]:
                kd, vd = kd * s["k_scales"][slots, h, :, None].double(), vd * s["v_scales"][slots, h, :, None].double()
            kd, vd = kd.reshape(-1, dim)[:n], vd.reshape(-1, dim)[:n]
            group = heads // kv
            for lo in range(0, new, 1024):  # a slab of the new tokens: their scores fit in memory
                hi = min(new, lo + 1024)
                pos = torch.arange(n - new + lo, n - new + hi, device=DEVICE)[:, None]
                key = torch.arange(n, device=DEVICE)[None]
                hidden = key > pos
                if case["window"]:
                    hidden = hidden | (key <= pos - case["window"])
                for g in range(h * group, (h + 1) * group):
                    score = (s["q"][first + lo: first + hi, g].double() @ kd.T * s["scale"]).masked_fill(hidden, -math.inf)
                    lse[first + lo: first + hi, g] = torch.logsumexp(score, -1)
                    out[first + lo: first + hi, g] = torch.softmax(score, -1) @ vd
        first += new
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}
