"""Products with an epilogue, the choice of experts and the sum over them, against
their definitions in float64 (the weights' values from the oracle).

Tolerances. A product's sum may be off by B = 1e-2 |w| |x| / sqrt(k) (the product's
contract). An activation with slope at most L = 1.13 (silu 1.10, both gelus 1.13; a silu of any
alpha > 0 has silu's, since silu_a(v) = silu(a v) / a) carries it on as L B; a gate a(g) u gives
L B_g |u| + |a(g)| B_u + L B_g B_u (clamps have slope at most 1). The activations' own forms
are off by less than 2^-16 of their value, float32's other roundings by less still, and the
result is rounded once to bfloat16: 2^-8 of it.
"""
import math

import numpy as np
import pytest
import torch

import oracle
import packed_qmatmul_gb300 as qm
from packed_qmatmul_gb300 import synth
from wutil import to_oracle

pytestmark = pytest.mark.gpu

SLOPE = {None: 1.0, "relu": 1.0, "silu": 1.13, "gelu": 1.13, "gelu_tanh": 1.13}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from packed_qmatmul_gb300 import build

    build.build()
    qm.load_library()
    torch.cuda.set_device(0)


def make(kind, seed, n, k, lead=()):
    """A packed weight whose products with unit activations are about 1 in size, and its values in float64."""
    g = synth.rng(seed)
    size = k ** -0.5
    if kind.startswith("affine"):
        bits, gs = int(kind[6]), int(kind.split("_g")[1])
        w = synth.affine_weight(g, n, k, bits=bits, group_size=gs, lead=lead, scale_sigma=2 * size / (1 << bits), bias_sigma=size / 2)
    elif kind == "q8_0":
        w = synth.q8_0_weight(g, n, k, lead=lead, d_sigma=size / 73)
    elif kind in ("mxfp4", "mxfp4_blocks"):
        lo = 127 + round(math.log2(size)) - 3
        w = (synth.mxfp4_weight if kind == "mxfp4" else synth.mxfp4_blocks_weight)(g, n, k, lead=lead, scale_lo=lo, scale_hi=lo + 2)
    elif kind == "q4_k":
        w = synth.q4_k_weight(g, n, k, lead=lead, d_sigma=size / 300)
    else:
        w = synth.q6_k_weight(g, n, k, lead=lead, d_sigma=size / 1500)
    values = torch.from_numpy(oracle.dequant(to_oracle(w), oracle.F32).astype(np.float64).reshape(*lead, n, k)).cuda()
    return qm.QWeight.from_arrays(w, flags=qm.QM_WEIGHT_STATIC), values


def randn(seed, *shape, dtype=torch.bfloat16):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


def act64(act, v, alpha=1.0):
    if act == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if act == "silu":
        return v / (1 + torch.exp(-alpha * v))
    if act == "gelu":
        return v * torch.erfc(-v / math.sqrt(2)) / 2
    if act == "gelu_tanh":
        return v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))) / 2
    return v


def expected(values, x, bias, ep, residual):
    """(y, how far off it may be) in float64, for x [M, k] and values [n, k] (or [M, n, k])."""
    k = values.shape[-1]
    v = torch.einsum("mk,nk->mn" if values.dim() == 2 else "mk,mnk->mn", x.double(), values)
    b = 1e-2 * x.double().norm(dim=1)[:, None] * values.norm(dim=-1) / math.sqrt(k)
    if bias is not None:
        v = v + bias.double()
    act, alpha, limit = ep.act, ep._tail[3], ep._tail[4] or math.inf
    slope = SLOPE[act]
    if ep.gated:
        g, u = v[:, 0::2].clamp(max=limit), v[:, 1::2].clamp(-limit, limit) + ep._tail[5]
        bg, bu = b[:, 0::2], b[:, 1::2]
        a = act64(act, g, alpha)
        y, off = a * u, slope * bg * u.abs() + a.abs() * bu + slope * bg * bu
    else:
        y, off = act64(act, v, alpha), slope * b
    off = off + 2.0 ** -16 * y.abs()
    if residual is not None:
        y = y + residual.double()
    return y, off + 2.0 ** -8 * (y.abs() + off)


def check(got, want, off, what=""):
    d = (got.double() - want).abs()
    bad = ~(d <= off)
    assert not bad.any(), (what, int(bad.sum()), d[bad][:4].tolist(), off[bad][:4].tolist(), bad.nonzero()[:4].tolist())


# Every kernel a product can take: (format, n, k, M).
PRODUCTS = (
    # one token, rows in registers: every format, k in one, two, four chunks, an odd count of chunks
    [(kind, 300, 1024, 1) for kind in ("affine2_g64", "affine3_g64", "affine4_g32", "affine5_g64", "affine6_g128", "affine8_g64", "q8_0", "mxfp4",
                                       "mxfp4_blocks", "q4_k", "q6_k")]
    + [("affine4_g64", 258, 2048, 1), ("affine4_g64", 34, 4096, 1), ("affine4_g64", 2, 5120, 1), ("mxfp4", 130, 96, 1)]
    # one token of a weight past 24 MB: the tensor-map pipeline
    + [("q8_0", 6200, 4096, 1), ("affine4_g64", 12002, 4096, 1)]
    # a few tokens in registers: k split and not
    + [("affine4_g64", 210, 512, 2), ("affine4_g128", 66, 4096, 8), ("affine4_g32", 1030, 1024, 5), ("affine4_g64", 18, 256, 3)]
    # the tensor-map pipeline: k whole and split over a cluster, more than one stage
    + [("affine4_g32", 1002, 1600, 5), ("affine8_g64", 70, 4096, 16), ("q8_0", 130, 4096, 3), ("q8_0", 9000, 512, 9), ("mxfp4", 2882, 2880, 4),
       ("mxfp4_blocks", 514, 1024, 16), ("mxfp4", 6, 64, 2)]
    # tensor cores: one and several token tiles, k split, ragged rows and columns
    + [("affine4_g64", 1002, 512, 17), ("affine3_g64", 514, 1024, 33), ("q8_0", 390, 4096, 77), ("mxfp4", 2880, 2880, 128), ("mxfp4", 262, 736, 129),
       ("mxfp4_blocks", 136, 1024, 300), ("q4_k", 200, 512, 257), ("affine8_g32", 4098, 256, 600), ("q8_0", 64, 8192, 40)]
    # the plain kernel
    + [("q6_k", 70, 512, 5), ("q4_k", 70, 256, 3), ("q6_k", 18, 256, 40), ("affine5_g32", 30, 96, 9)]
)


@pytest.mark.parametrize("kind,n,k,M", PRODUCTS)
def test_fused_against_the_definition(kind, n, k, M):
    w, values = make(kind, 7, n, k)
    x = randn(1, M, k)
    plain = qm.apply(w, x)
    for i, (act, dtype, gated, with_res) in enumerate([(None, torch.bfloat16, False, True), ("silu", None, False, False), ("gelu", torch.float32, False, True),
                                                       ("gelu_tanh", torch.float16, False, False), ("silu", torch.bfloat16, True, True),
                                                       ("gelu_tanh", None, True, False), (None, torch.float32, True, False)]):
        bias = None if dtype is None else randn(2 + i, n, dtype=dtype)
        clamps = dict(limit=1.5, up_offset=1.0, alpha=1.702) if act == "silu" and gated else {}
        ep = qm.Epilogue(bias=bias, act=act, gated=gated, **clamps)
        cols = n // 2 if gated else n
        res = randn(20 + i, M, cols) if with_res else None
        y = qm.apply_fused(w, x, ep, res)
        assert y.shape == (M, cols)
        check(y, *expected(values, x, bias, ep, res), what=(act, gated))
        assert torch.equal(y, qm.apply_fused(w, x, ep, res))  # the same bits again
    # rounding keeps order, and the sums are the same: relu before it is relu after it; nothing is nothing
    assert torch.equal(qm.apply_fused(w, x, qm.Epilogue(act="relu")), torch.relu(plain) + 0.0)
    assert torch.equal(qm.apply_fused(w, x, qm.Epilogue()), plain)
    qm.qm_device_status()


@pytest.mark.parametrize("kind,n,k,M", [("affine4_g64", 301, 1024, 1), ("affine4_g64", 37, 512, 4), ("q8_0", 131, 1024, 7), ("mxfp4", 1001, 512, 30),
                                        ("affine4_g64", 77, 2048, 200), ("q6_k", 9, 256, 3)])
def test_odd_rows(kind, n, k, M):
    w, values = make(kind, 8, n, k)
    x, bias, res = randn(3, M, k), randn(4, n, dtype=torch.float32), randn(5, M, n)
    ep = qm.Epilogue(bias=bias, act="silu")
    check(qm.apply_fused(w, x, ep, res), *expected(values, x, bias, ep, res))


@pytest.mark.parametrize("M", [1, 2, 12, 40, 300])
def test_residual_strides_and_in_place(M):
    n, k = 264, 512
    w, values = make("affine4_g64", 9, n, k)
    x = randn(6, M, k)
    ep = qm.Epilogue(act="gelu")
    wide = randn(7, M, n + 21)
    want = qm.apply_fused(w, x, ep, wide[:, 5:5 + n].contiguous())  # an odd offset and stride
    assert torch.equal(qm.apply_fused(w, x, ep, wide[:, 5:5 + n]), want)
    even = randn(7, M, n + 20)
    assert torch.equal(qm.apply_fused(w, x, ep, even[:, 2:2 + n]), qm.apply_fused(w, x, ep, even[:, 2:2 + n].contiguous()))
    one = randn(8, 1, n)
    assert torch.equal(qm.apply_fused(w, x, ep, one.expand(M, n)), qm.apply_fused(w, x, ep, one.repeat(M, 1)))
    y = torch.empty(M, n, dtype=torch.bfloat16, device="cuda").copy_(wide[:, 5:5 + n])  # its own, aligned
    qm.qm_apply_fused(w, x, ep, y, residual=y)
    assert torch.equal(y, want)
    gate = qm.Epilogue(act="silu", gated=True)
    y = randn(9, M, n // 2)
    want = qm.apply_fused(w, x, gate, y.clone())
    qm.qm_apply_fused(w, x, gate, y, residual=y)
    assert torch.equal(y, want)


@pytest.mark.parametrize("M", [1, 5, 12])
def test_rows_past_the_last_do_not_decide(M):
    """A ragged last stage's missing rows hold what an earlier launch left in shared memory: whatever that is, the
    rows beside them are summed the same way. k = 1600 keeps whole rows of scales in a stage; the launches between
    leave scales of every size there."""
    n, k = 33002 if M == 1 else 1002, 1600  # one token: a weight past 24 MB, for the tensor-map pipeline
    w = qm.QWeight.from_arrays(synth.affine_weight(synth.rng(5), n, k, bits=4, group_size=32))
    x = torch.randn(M, k, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    want = None
    for scale in (0.0, 1.0, 2.0 ** 100, float("inf"), float("nan"), 2.0 ** -100):
        fill = synth.affine_weight(synth.rng(7), (n + 31) // 32 * 32, k, bits=4, group_size=32)
        f = qm.QWeight.from_arrays(fill)
        f.scales.view(torch.bfloat16).fill_(scale)
        f.biases.view(torch.bfloat16).fill_(scale)
        qm.apply(f, x)
        y = qm.apply(w, x)
        want = y if want is None else want
        assert torch.equal(y, want), scale


def test_exact_sums_round_once():
    """Zero products: bias, activation and residual alone, rounded once."""
    n, k = 256, 256
    w, _ = make("affine4_g64", 10, n, k)
    bias = randn(11, n, dtype=torch.float32)
    for M in (1, 4, 16, 64, 260):
        x, res = torch.zeros(M, k, dtype=torch.bfloat16, device="cuda"), randn(12, M, n)
        y = qm.apply_fused(w, x, qm.Epilogue(bias=bias), res)
        assert torch.equal(y, (bias + res.float()).bfloat16())
        y = qm.apply_fused(w, x, qm.Epilogue(bias=bias, act="relu"), res)
        assert torch.equal(y, (bias.clamp(min=0) + res.float()).bfloat16())


def test_special_values():
    """Sums of every size, infinities and NaN through the activations (the bias carries them)."""
    inf, nan = math.inf, math.nan
    v = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 3.0, -3.0, 12.0, -12.0, 60.0, -60.0, 87.0, -87.0, 1e4, -1e4, 1e30, -1e30, inf, -inf, nan, -20.0], device="cuda")
    n = 2 * v.numel()
    bias = torch.cat([v, v.flip(0)])
    w, _ = make("affine4_g64", 13, n, 256)
    for M in (1, 3, 16, 50):
        x = torch.zeros(M, 256, dtype=torch.bfloat16, device="cuda")
        for act in ("relu", "silu", "gelu", "gelu_tanh"):
            y = qm.apply_fused(w, x, qm.Epilogue(bias=bias, act=act)).double()
            want = act64(act, bias.double())
            if act in ("gelu", "gelu_tanh"):  # the definition in float64 loses its tail past -8: formed apart
                tail = (bias < -8) & (bias > -1e3)
                assert (y[0][tail].abs() < 1e-10).all()
                want = torch.where(tail, y[0], want)
            want = want.expand(M, n)
            nans = torch.isnan(want)
            assert torch.equal(nans, torch.isnan(y)), act
            infs = torch.isinf(want)
            assert torch.equal(y[infs], want[infs]), act
            rest = ~nans & ~infs
            # one rounding of the value, or of bfloat16's smallest step where it is that small
            assert ((y - want)[rest].abs() <= want[rest].abs() * (2.0 ** -8 + 2.0 ** -14) + 2.0 ** -133).all(), act
        gate = qm.Epilogue(bias=bias, act="silu", gated=True, limit=7.0, up_offset=1.0)
        y = qm.apply_fused(w, x, gate).double()
        g, u = bias[0::2].double(), bias[1::2].double()
        want = (act64("silu", g.clamp(max=7.0)) * (u.clamp(-7.0, 7.0) + 1.0)).expand(M, n // 2)
        assert torch.equal(torch.isnan(want), torch.isnan(y))
        rest = ~torch.isnan(want)
        assert ((y - want)[rest].abs() <= want[rest].abs() * (2.0 ** -8 + 2.0 ** -14) + 2.0 ** -133).all()


def test_empty_products():
    w = qm.QWeight("affine", (6, 0), torch.empty(6, 0, dtype=torch.uint8, device="cuda"), torch.empty(6, 0, dtype=torch.bfloat16, device="cuda"),
                   torch.empty(6, 0, dtype=torch.bfloat16, device="cuda"), bits=4, group_size=64)
    bias, res = randn(1, 6, dtype=torch.float32), randn(2, 3, 3)
    x = torch.empty(3, 0, dtype=torch.bfloat16, device="cuda")
    y = qm.apply_fused(w, x, qm.Epilogue(bias=bias, act=None, gated=True), res)
    # the gate's product is not rounded before the residual meets it
    assert torch.equal(y, (bias[0::2].double() * bias[1::2].double() + res.double()).bfloat16())
    assert torch.equal(qm.apply_fused(w, x, qm.Epilogue()), torch.zeros(3, 6, dtype=torch.bfloat16, device="cuda"))
    w, _ = make("affine4_g64", 1, 8, 64)
    assert qm.apply_fused(w, randn(1, 0, 64), qm.Epilogue(act="silu")).shape == (0, 8)


# ---------------------------------------------------------------- experts
EXPERTS = [
    # (format, E, n, k, T, topk): decode chunks, k split, tensor-core tiles of 128 and of 256, the plain kernel
    ("mxfp4", 8, 192, 288, 3, 2), ("affine4_g64", 5, 144, 512, 11, 3), ("q8_0", 4, 64, 4096, 2, 1), ("mxfp4", 32, 576, 288, 64, 4),
    ("mxfp4", 4, 320, 288, 100, 3), ("affine4_g32", 3, 130, 256, 200, 2), ("mxfp4", 2, 262, 288, 700, 2), ("q4_k", 2, 34, 256, 90, 2),
    ("q6_k", 3, 10, 256, 7, 2), ("affine3_g64", 3, 34, 128, 5, 2),
]


@pytest.mark.parametrize("kind,E,n,k,T,topk", EXPERTS)
def test_experts_fused_against_the_definition(kind, E, n, k, T, topk):
    w, values = make(kind, 14, n, k, (E,))
    gen = torch.Generator(device="cuda").manual_seed(15)
    ids = torch.randint(0, E, (T, topk), generator=gen, device="cuda")
    ids.view(-1)[1::5] = -1
    ids.view(-1)[3::7] = E
    if T > 4:
        ids[T // 2:][ids[T // 2:] == 0] = 1  # an expert that half the tokens leave out
    P = T * topk
    flat = ids.view(-1)
    live = (flat >= 0) & (flat < E)
    for i, (act, dtype, gated, per, itype) in enumerate([("silu", torch.bfloat16, True, False, torch.int32), ("gelu", torch.float32, False, True, torch.int64),
                                                         (None, torch.float16, False, False, torch.int32), ("gelu_tanh", None, True, True, torch.int32)]):
        x = randn(16 + i, P if per else T, k)
        x.view(-1, k)[0] *= 30.0  # a row of another size
        bias = None if dtype is None else randn(30 + i, E, n, dtype=dtype)
        clamps = dict(limit=1.5, up_offset=1.0, alpha=1.702) if act == "silu" else {}
        ep = qm.Epilogue(bias=bias, act=act, gated=gated, **clamps)
        y = qm.apply_experts_fused(w, ids.to(itype), x, ep).view(P, -1)
        rows = x if per else x.repeat_interleave(topk, 0)
        assert (y[~live] == 0).all()
        for e in range(E):
            at = (flat == e).nonzero()[:, 0]
            if at.numel():
                check(y[at], *expected(values[e], rows[at], None if bias is None else bias[e], ep, None), what=(act, e))
    assert torch.equal(qm.apply_experts_fused(w, ids, x, qm.Epilogue(act="relu")), torch.relu(qm.apply_experts(w, ids, x)) + 0.0)
    assert torch.equal(qm.apply_experts_fused(w, ids, x, qm.Epilogue()), qm.apply_experts(w, ids, x))
    qm.qm_device_status()


def test_experts_without_positions():
    w, _ = make("mxfp4", 14, 64, 64, (4,))
    ep = qm.Epilogue(bias=randn(1, 4, 64), act="silu")
    assert qm.apply_experts_fused(w, torch.empty(0, 2, dtype=torch.int32, device="cuda"), randn(2, 0, 64), ep).shape == (0, 2, 64)
    y = qm.apply_experts_fused(w, torch.full((3, 2), -1, dtype=torch.int32, device="cuda"), randn(2, 3, 64), ep)
    assert (y == 0).all()


def test_experts_of_empty_sums():
    E, n = 3, 6
    w = qm.QWeight("affine", (E, n, 0), *(torch.empty(E, n, 0, dtype=d, device="cuda") for d in (torch.uint8, torch.bfloat16, torch.bfloat16)), bits=4,
                   group_size=64)
    bias = randn(1, E, n, dtype=torch.float32)
    ids = torch.tensor([[0, 2], [1, 5]], dtype=torch.int32, device="cuda")
    y = qm.apply_experts_fused(w, ids, torch.empty(2, 0, dtype=torch.bfloat16, device="cuda"), qm.Epilogue(bias=bias, act="relu"))
    want = bias.clamp(min=0).bfloat16()
    assert torch.equal(y[0, 0], want[0]) and torch.equal(y[0, 1], want[2]) and torch.equal(y[1, 0], want[1]) and (y[1, 1] == 0).all()


# ---------------------------------------------------------------- the choice of experts
def select64(logits, topk, score="softmax", bias=None, groups=1, topk_groups=None, group_score="max", renormalize=True, scale=1.0):
    """ids and weights by the definition, token by token in float64."""
    topk_groups = groups if topk_groups is None else topk_groups
    x = logits.double().cpu().numpy()
    T, E = x.shape
    b = np.zeros(E) if bias is None else bias.double().cpu().numpy()
    ids, weights = np.full((T, topk), -1, np.int32), np.zeros((T, topk))
    size = E // groups
    for t in range(T):
        row = x[t]
        if score == "softmax":
            if np.isnan(row).any() or np.isposinf(row).any():
                weights[t] = np.nan
                continue
            if np.isneginf(row).all():
                continue
            e = np.exp(row - row.max())
            s = e / e.sum()
        else:
            with np.errstate(over="ignore"):
                s = 1 / (1 + np.exp(-row))
        # without a bias the logits are in the scores' order, and distinct where float64's scores may not be
        key = s + b if bias is not None else row.copy()
        gkey = s + b
        hidden = ~(row > -np.inf) | ~(b > -np.inf) | np.isnan(key)
        key[hidden] = -np.inf
        gkey[hidden] = -np.inf
        if groups > 1:
            best = []
            for g in range(groups):
                part = np.sort((key if group_score == "max" else gkey)[g * size:(g + 1) * size])[::-1]
                best.append(part[0] if group_score == "max" else part[0] + part[1])
            kept = sorted(range(groups), key=lambda g: (-best[g], g))[:topk_groups]
            for g in range(groups):
                if g not in kept:
                    key[g * size:(g + 1) * size] = -np.inf
        order = sorted((i for i in range(E) if key[i] > -np.inf), key=lambda i: (-key[i], i))[:topk]
        if order:
            ids[t, :len(order)] = order
            got = s[order]
            if renormalize:
                if score == "sigmoid":  # in the logarithm, where scores are too small to add
                    ls = -np.logaddexp(0, -row[order])
                    got = np.exp(ls - ls.max())
                    got = got / got.sum()
                else:
                    got = np.exp(row[order] - row[order].max())
                    got = got / got.sum()
            weights[t, :len(order)] = got * scale
    return ids, weights


def check_select(logits, topk, bias=None, **kw):
    ids, weights = qm.experts_select(logits, qm.Router(topk, bias=bias, **kw))
    want_ids, want = select64(logits, topk, bias=bias, **kw)
    assert ids.dtype == torch.int32 and weights.dtype == torch.float32
    np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
    got = weights.double().cpu().numpy()
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    fine = ~np.isnan(want)
    # exp's argument is rounded by 2^-24 of its size (below 104), its value by 2^-22, sums of at most 1024
    # terms as a tree of 37 by 37 * 2^-24, the quotient and the scale by 2^-24 each: less than 2^-16 in all
    assert (np.abs(got - want)[fine] <= 2.0 ** -16 * np.abs(want[fine]) + 2.0 ** -140).all()
    return ids, weights


SELECTS = [
    dict(E=32, topk=4), dict(E=1, topk=1), dict(E=7, topk=7), dict(E=33, topk=2, renormalize=False), dict(E=128, topk=8, scale=2.5),
    dict(E=1000, topk=31), dict(E=1024, topk=10, score="sigmoid"), dict(E=64, topk=6, score="sigmoid", bias=True),
    dict(E=64, topk=6, bias=True), dict(E=512, topk=22, bias=True, score="sigmoid", scale=5.0),
    dict(E=256, topk=8, score="sigmoid", bias=True, groups=8, topk_groups=4, group_score="top2", scale=2.5),
    dict(E=160, topk=6, groups=8, topk_groups=3, renormalize=False, scale=16.0), dict(E=72, topk=5, groups=3, topk_groups=2, group_score="top2"),
    dict(E=100, topk=30, groups=5, topk_groups=1), dict(E=96, topk=4, groups=32, topk_groups=7, score="sigmoid", group_score="top2"),
    dict(E=64, topk=3, groups=4, topk_groups=4, group_score="top2", bias=True), dict(E=960, topk=9, groups=6, topk_groups=2, bias=True, score="sigmoid"),
    dict(E=1020, topk=8, groups=17, topk_groups=4, score="sigmoid", group_score="top2"), dict(E=12, topk=3, groups=12, topk_groups=2), dict(E=544, topk=5, groups=17, topk_groups=3, bias=True, group_score="top2"),
]


@pytest.mark.parametrize("kw", SELECTS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_select_against_the_definition(kw, dtype):
    kw = dict(kw)
    E, topk = kw.pop("E"), kw.pop("topk")
    bias = randn(41, E, dtype=torch.float32) * 0.1 if kw.pop("bias", False) else None
    for T in (1, 5, 77):
        wide = randn(42 + T, T, E + 3, dtype=torch.float32).to(dtype) * 2
        check_select(wide[:, 1:1 + E], topk, bias=bias, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_select_ties_and_near_ties(score):
    gen = torch.Generator(device="cuda").manual_seed(50)
    T, E = 40, 256
    few = torch.randint(-2, 3, (T, E), generator=gen, device="cuda").bfloat16()  # many equal logits
    zero = torch.zeros(E, device="cuda")
    steps = torch.randint(-2, 3, (E,), generator=gen, device="cuda").float() / 8
    for kw in (dict(), dict(groups=8, topk_groups=3), dict(groups=8, topk_groups=3, group_score="top2")):
        check_select(few, 9, score=score, **kw)
        check_select(few, 9, score=score, bias=zero, **kw)
        check_select(torch.zeros(T, E, device="cuda"), 9, score=score, bias=zero, **kw)
        check_select(torch.zeros(T, E, device="cuda"), 9, score=score, **kw)
        # scores that float32 cannot tell apart: logits 1e-6 wide, and biases that meet them
        check_select(randn(51, T, E, dtype=torch.float32) * 1e-6, 9, score=score, bias=zero, **kw)
        check_select(randn(51, T, E, dtype=torch.float32) * 1e-6, 9, score=score, bias=randn(52, E, dtype=torch.float32) * 1e-7, **kw)
        check_select(randn(53, T, E, dtype=torch.float32) * 1e-4, 9, score=score, **kw)
        # saturated and vanishing scores
        check_select(randn(54, T, E, dtype=torch.float32) * 2 + 30, 9, score=score, **kw)
        check_select(randn(55, T, E, dtype=torch.float32) * 3 - 90, 9, score=score, **kw)
        check_select(randn(55, T, E, dtype=torch.float32) * 3 - 90, 9, score=score, bias=zero, **kw)
        check_select(few, 9, score=score, bias=steps, renormalize=False, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups", [dict(), dict(groups=4, topk_groups=2), dict(groups=4, topk_groups=2, group_score="top2")])
def test_select_masks_and_what_is_not_finite(score, biased, groups):
    T, E = 12, 48
    x = randn(60, T, E, dtype=torch.float32)
    x[0] = -math.inf                      # nothing to choose from
    x[1, 3:] = -math.inf                  # fewer than topk
    x[2, ::2] = -math.inf
    x[3, 5] = math.nan
    x[4, 7] = math.inf
    x[5] = torch.finfo(torch.float32).min
    x[6, 4:] = torch.finfo(torch.float32).min
    x[7] = math.nan
    x[8, :47] = -math.inf
    x[9, 30:] = -math.inf
    x[10] = 3.0e38
    bias = None
    if biased:
        bias = randn(61, E, dtype=torch.float32) * 0.2
        bias[9] = -math.inf
        bias[20] = -math.inf
    for renormalize in (True, False):
        check_select(x, 6, score=score, bias=bias, renormalize=renormalize, **groups)


def test_select_of_many_tokens_and_outputs():
    T, E = 9001, 64
    x = randn(62, T, E, dtype=torch.float32)
    ids, weights = check_select(x, 4)
    out = torch.full((T + 2, 4), 77, dtype=torch.int32, device="cuda"), torch.full((T + 2, 4), 7.0, device="cuda")
    qm.qm_experts_select(x, qm.Router(4), out[0][1:-1], out[1][1:-1])
    assert torch.equal(out[0][1:-1], ids) and torch.equal(out[1][1:-1], weights)
    assert (out[0][[0, -1]] == 77).all() and (out[1][[0, -1]] == 7.0).all()
    assert qm.experts_select(x[:0], qm.Router(4))[0].shape == (0, 4)


# ---------------------------------------------------------------- the sum over a token's experts
@pytest.mark.parametrize("T,topk,n", [(1, 4, 2880), (3, 1, 8), (5, 8, 1001), (7, 3, 24), (2, 31, 40), (300, 6, 512), (1, 0, 16), (9, 5, 7), (2000, 4, 1016), (33, 9, 1002),
                                      (11, 2, 1), (6, 4, 13), (5, 17, 2003)])
def test_combine_against_the_definition(T, topk, n):
    y, w = randn(70, T, topk, n), torch.rand(T, topk, device="cuda") - 0.3
    wide = randn(71, T, n + 8)
    for res in (None, randn(72, T, n), wide[:, 8:], wide[:, 3:3 + n], randn(73, 1, n).expand(T, n)):
        got = qm.experts_combine(y, w, res)
        want = (y.double() * w.double()[..., None]).sum(1)
        size = (y.double() * w.double()[..., None]).abs().sum(1)
        if res is not None:
            want, size = want + res.double(), size + res.double().abs()
        # each of topk + 1 additions by 2^-24 of what is summed so far, then one rounding
        assert ((got.double() - want).abs() <= (topk + 1) * 2.0 ** -24 * size * 1.01 + 2.0 ** -8 * want.abs() + 2.0 ** -140).all()
    out = randn(72, T, n)
    want = qm.experts_combine(y, w, out.clone())
    qm.qm_experts_combine(y, w, out, residual=out)
    assert torch.equal(out, want)


@pytest.mark.parametrize("n", [8, 9, 15, 1001])
def test_combine_writes_its_rows_alone(n):
    """Buffers cut from the middle of larger ones: nothing beside the rows is written, NaN beside y's is not read."""
    T, topk = 5, 3
    y = torch.full((T * topk * n + 64,), math.nan, dtype=torch.bfloat16, device="cuda")
    y[32:32 + T * topk * n] = randn(75, T * topk * n)
    out = torch.full((T * n + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    w = torch.rand(T, topk, device="cuda")
    body = y[32:32 + T * topk * n].view(T, topk, n)
    qm.qm_experts_combine(body, w, out[32:32 + T * n].view(T, n))
    assert torch.equal(out[32:32 + T * n].view(T, n), qm.experts_combine(body.clone(), w)) and torch.isfinite(out).all()
    assert (out[:32] == 7.0).all() and (out[32 + T * n:] == 7.0).all()


def test_combine_passes_on_what_is_not_finite():
    y, w = randn(74, 4, 2, 64), torch.rand(4, 2, device="cuda") + 0.1
    y[0, 1, 3] = math.inf
    y[1, 0, 5] = math.nan
    w[2, 0] = math.nan
    w[3] = 0.0
    got = qm.experts_combine(y, w)
    assert got[0, 3] == math.inf and torch.isnan(got[1, 5]) and torch.isnan(got[2]).all() and (got[3] == 0).all()
    assert torch.isfinite(got).sum() == 4 * 64 - 2 - 64
    assert qm.experts_combine(y[:0], w[:0]).shape == (0, 64)


# ---------------------------------------------------------------- together
class Experts:
    """A layer of experts: the choice, gate and up rows in turn, down, and the sum added to the hidden state."""

    def __init__(self, E=16, hidden=256, inner=320, topk=4):
        self.up, self.up_values = make("mxfp4", 80, 2 * inner, hidden, (E,))
        self.down, self.down_values = make("mxfp4", 81, hidden, inner, (E,))
        self.up_bias, self.down_bias = randn(82, E, 2 * inner) * 0.3, randn(83, E, hidden) * 0.3
        self.router = qm.Router(topk, score="sigmoid", bias=randn(84, E, dtype=torch.float32) * 0.1, groups=4, topk_groups=2, group_score="top2", scale=1.5)
        self.gate = qm.Epilogue(bias=self.up_bias, act="silu", gated=True, alpha=1.702, limit=7.0, up_offset=1.0)
        self.back = qm.Epilogue(bias=self.down_bias)

    def __call__(self, x, logits, stream=None):
        ids, weights = qm.experts_select(logits, self.router, stream=stream)
        inner = qm.apply_experts_fused(self.up, ids, x, self.gate, stream=stream)
        T, topk, n = inner.shape
        y = qm.apply_experts_fused(self.down, ids, inner.view(T * topk, n), self.back, stream=stream)
        return qm.experts_combine(y, weights, x, stream=stream)

    def check(self, x, logits, got):
        r = self.router
        ids, weights = select64(logits, r.topk, score="sigmoid", bias=r.bias, groups=4, topk_groups=2, group_score="top2", scale=1.5)
        want, off = x.double(), torch.zeros(x.shape, device="cuda", dtype=torch.float64)
        for j in range(r.topk):
            e = torch.from_numpy(ids[:, j]).long().cuda()
            w = torch.from_numpy(weights[:, j]).cuda()[:, None]
            a, a_off = expected(self.up_values[e], x, self.up_bias[e], self.gate, None)
            v, v_off = expected(self.down_values[e], a, self.down_bias[e], self.back, None)
            v_off = v_off + torch.einsum("mk,mnk->mn", a_off, self.down_values[e].abs())
            want, off = want + w * v, off + w * v_off
        check(got, want, off + 2.0 ** -8 * (want.abs() + off) + 1e-5)


@pytest.mark.parametrize("T", [1, 5, 200])
def test_layer_of_experts(T):
    layer = Experts()
    x, logits = randn(90, T, 256), randn(91, T, 16)
    layer.check(x, logits, layer(x, logits))


def test_layer_of_experts_on_a_stream_and_replayed():
    layer = Experts()
    T = 24
    x, logits = randn(92, T, 256), randn(93, T, 16)
    plain = layer(x, logits)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = layer(x, logits, stream=side)
    side.synchronize()
    assert torch.equal(got, plain)
    with torch.cuda.stream(side):
        layer(x, logits)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x, logits)
    for seed in (94, 95):
        x.copy_(randn(seed, T, 256))
        logits.copy_(randn(seed + 10, T, 16))
        logits[3] = -math.inf  # a token that no expert takes keeps its hidden state
        layer.router.bias.copy_(randn(seed + 20, 16, dtype=torch.float32) * 0.1)
        graph.replay()
        assert torch.equal(out, layer(x, logits))
        assert torch.equal(out[3], x[3])
        some = [t for t in range(T) if t != 3]
        layer.check(x[some], logits[some], out[some])
    qm.qm_device_status()


def test_two_streams_at_once():
    """Layers on two streams, each with its own workspaces, give what they give alone."""
    layer = Experts()
    xs = [randn(96 + i, 40, 256) for i in range(2)]
    ls = [randn(98 + i, 40, 16) for i in range(2)]
    want = [layer(x, l) for x, l in zip(xs, ls)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(layer(xs[i], ls[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


def test_gates_laid_out_by_take():
    """A weight whose gates and ups lie in halves, its packed rows taken in pairs once."""
    n, k, M = 192, 512, 20
    w, values = make("affine4_g64", 100, n, k)
    order = torch.arange(n, device="cuda").view(2, n // 2).T.reshape(-1).to(torch.int32)
    pairs, _ = qm.take(w, 0, order)
    x = randn(101, M, k)
    ep = qm.Epilogue(act="silu", gated=True)
    check(qm.apply_fused(pairs, x, ep), *expected(values[order.long()], x, None, ep, None))


def test_tensors_of_another_gpu_than_the_current_one(monkeypatch):
    w, _ = make("affine4_g64", 1, 8, 64)
    experts, _ = make("mxfp4", 2, 64, 64, (4,))
    ids = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    monkeypatch.setattr(qm, "_device", lambda: 1)
    for call in (lambda: qm.apply_fused(w, randn(1, 3, 64), qm.Epilogue(act="silu")), lambda: qm.apply_experts_fused(experts, ids, randn(1, 3, 64), qm.Epilogue()),
                 lambda: qm.experts_select(randn(1, 3, 16), qm.Router(2)), lambda: qm.experts_combine(randn(1, 3, 2, 8), torch.ones(3, 2, device="cuda"))):
        with pytest.raises(qm.QMError, match="device"):
            call()


# ---------------------------------------------------------------- where calls go wrong
def same(a, b):
    """Equal, with every NaN equal to every other."""
    nan = torch.isnan(a)
    return torch.equal(nan, torch.isnan(b)) and torch.equal(a[~nan], b[~nan])


@pytest.mark.parametrize("M", [1, 3, 12, 40, 200])
def test_activations_that_are_not_finite(M):
    """Infinite and NaN activations: what the plain product gives, through relu and an added row."""
    w, _ = make("affine4_g64", 110, 130, 512)
    x = randn(111, M, 512)
    x[0, 3] = math.inf
    if M > 1:
        x[1, 9] = math.nan
        x[-1, 11] = -math.inf
    plain, res = qm.apply(w, x), randn(112, 1, 130).expand(M, 130)
    y = qm.apply_fused(w, x, qm.Epilogue(act="relu"))
    assert same(y, torch.relu(plain) + 0.0)
    y = qm.apply_fused(w, x, qm.Epilogue(), res)
    odd = ~torch.isfinite(plain)
    assert odd.any() and same(y[odd], plain[odd])
    assert torch.isfinite(y[~odd]).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [dict(), dict(groups=4, topk_groups=2), dict(groups=4, topk_groups=2, group_score="top2")])
def test_select_with_a_bias_that_is_not_finite(score, groups):
    x = randn(113, 9, 64, dtype=torch.float32)
    bias = randn(114, 64, dtype=torch.float32) * 0.1
    bias[[5, 21]] = math.inf
    bias[40] = math.nan
    bias[[50, 51, 52]] = -math.inf
    bias[33] = 1e30
    check_select(x, 7, score=score, bias=bias, **groups)
    check_select(x, 7, score=score, bias=torch.full((64,), -math.inf, device="cuda"), **groups)


def test_past_two_to_the_31_elements():
    """Offsets that 32 bits do not hold, in each of the calls; rows at the ends and about the border are looked at."""
    T, topk, n = 93_300, 8, 2880
    y = torch.empty(T, topk, n, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(115))
    w = torch.rand(T, topk, device="cuda")
    out = qm.experts_combine(y, w)
    at = torch.tensor([0, 1, (1 << 31) // (topk * n), (1 << 31) // (topk * n) + 1, T - 1], device="cuda")
    assert torch.equal(out[at], qm.experts_combine(y[at].contiguous(), w[at].contiguous()))
    del y, out
    T, E = 2_100_000, 1024
    logits = torch.empty(T, E, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(116))
    router = qm.Router(4)
    ids, weights = qm.experts_select(logits, router)
    at = torch.tensor([0, (1 << 31) // E - 1, (1 << 31) // E, T - 1], device="cuda")
    few = qm.experts_select(logits[at].contiguous(), router)
    assert torch.equal(ids[at], few[0]) and torch.equal(weights[at], few[1])
    del logits, ids, weights
    M, n, k = 150_100, 14336, 64
    wq, _ = make("mxfp4", 117, n, k)
    x, res = randn(118, M, k), torch.empty(M, n, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(119))
    ep = qm.Epilogue(act="silu")
    at = torch.tensor([0, (1 << 31) // n, (1 << 31) // n + 1, M - 1], device="cuda").repeat_interleave(80)  # 320 rows: the same kernel
    want = qm.apply_fused(wq, x[at].contiguous(), ep, res[at].contiguous())
    qm.qm_apply_fused(wq, x, ep, res, residual=res)
    assert torch.equal(res[at], want)
    qm.qm_device_status()
