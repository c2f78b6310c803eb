"""Head norms with rotation, the paged cache's append and the attention over it,
against their definitions in 64 bits.

Tolerances, from the arithmetic the operators state (sums and products in
float32, one rounding of the result): a result has to lie between the roundings
to its type of the exact value less and plus e. u is the type's unit roundoff, 2^-8 for
bfloat16 and 2^-11 for float16.

* head_norm_rope, cache_append: e is 2^-18 of the two products a rotated element
  is the difference of: the norm's factor is a sum of at most 256 squares (their
  roundings add up to a few 2^-24 of it) under a reciprocal root.
* cache_attend: a score's float32 sum of `dim` products is off by at most
  (dim + 4) 2^-23 of sum |q_i k_i| scale, which turns each weight by that factor
  twice (its own and the total's); a weight enters its product rounded to 16
  bits, a relative u each; so e is (u + 2 ds + 2^-16) sum_j w_j |v_j|, and the log-sum-exp within ds + 2^-20 (1 + |lse|).
"""
import math

import numpy as np
import pytest
import torch

import packed_qmatmul_gb300 as qm

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from packed_qmatmul_gb300 import build

    build.build()
    qm.load_library()
    torch.cuda.set_device(0)


def rounded_within(got, want, e):
    """Where got lies between the roundings of want - e and want + e to its type."""
    lo, hi = (want - e).to(got.dtype).double(), (want + e).to(got.dtype).double()
    return (got.double() >= lo) & (got.double() <= hi)


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.float32, sigma=1.0, mean=0.0):
    return (torch.randn(*shape, generator=g) * sigma + mean).to(dtype)


def angles(rows, dim, theta=1e4):
    at = torch.arange(rows, dtype=torch.float64)[:, None] * theta ** (-torch.arange(dim // 2, dtype=torch.float64) / max(dim // 2, 1))
    return torch.cat([at.cos(), at.sin()], 1).float()


# ---------------------------------------------------------------- definitions in 64 bits
def norm_rope_def(x, w, eps, table, pos, style):
    """(y, size): x [T, H, D] normed and turned, and the magnitudes a result's error scales with."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    if table is None:
        return y, y.abs()
    r = table.shape[1]
    inside = (pos >= 0) & (pos < table.shape[0])
    t = torch.where(inside[:, None], table.double()[pos.clamp(0, table.shape[0] - 1).long()], torch.zeros((), dtype=torch.float64))
    c, s = t[:, None, : r // 2], t[:, None, r // 2:]
    ia = torch.arange(r // 2) if style == "half" else torch.arange(0, r, 2)
    ib = ia + (r // 2 if style == "half" else 1)
    a, b = y[..., ia], y[..., ib]
    out, size = y.clone(), y.abs()
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia], size[..., ib] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    return out, size


def attend_def(q, keys, vals, new, length, group, scale, window, cap):
    """One sequence: q [new, H, D], keys and vals [length, KV, D] in 64 bits. out, lse, sum w |v|, score size."""
    H, D = q.shape[1:]
    out = torch.zeros(new, H, D, dtype=torch.float64)
    lse = torch.full((new, H), -math.inf, dtype=torch.float64)
    absv, size = torch.zeros_like(out), torch.zeros_like(lse)
    for i in range(new):
        p = length - new + i
        lo, hi = max(0, p - window + 1) if window else 0, min(p + 1, cap)
        if hi <= lo:
            continue
        k = keys[lo:hi].repeat_interleave(group, 1)  # [n, H, D]
        v = vals[lo:hi].repeat_interleave(group, 1)
        s = torch.einsum("hd,nhd->hn", q[i].double(), k) * scale
        lse[i] = torch.logsumexp(s, -1)
        w = torch.softmax(s, -1)
        out[i] = torch.einsum("hn,nhd->hd", w, v)
        absv[i] = torch.einsum("hn,nhd->hd", w, v.abs())
        size[i] = torch.einsum("hd,nhd->hn", q[i].double().abs(), k.abs()).amax(-1) * scale
    return out, lse, absv, size


# ---------------------------------------------------------------- a cache in any layout
class Paged:
    """Sequences' keys and values scattered over the pages of a cache on the GPU."""

    def __init__(self, g, seqs, kv, dim, page, dtype, codes=False, layout="heads", extra=2, fill=float("nan"), spare=1):
        self.seqs, self.kv, self.dim, self.page = seqs, kv, dim, page
        need = [-(-max(n, 0) // page) for _, n in seqs]
        self.width = max(max(need) + spare, 1)
        pages = sum(need) + extra
        order = torch.randperm(pages, generator=g)
        table = torch.full((len(seqs), self.width), -1, dtype=torch.int32)
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = order[at: at + n]
            at += n
        self.table = table
        store = torch.int8 if codes else dtype
        shape = (pages, kv, page, dim) if layout == "heads" else (pages, page, kv, dim)

        def parts():
            t = torch.full(shape, 0 if codes else fill, dtype=store)
            return t if layout == "heads" else t.permute(0, 2, 1, 3)

        self.k, self.v = parts(), parts()
        self.ks = torch.full((pages, kv, page), math.nan) if codes else None
        self.vs = torch.full((pages, kv, page), math.nan) if codes else None
        self.keys, self.vals = [], []
        for i, (_, n) in enumerate(seqs):
            n = max(n, 0)
            j = torch.arange(n)
            p, r = table[i].long()[j // page], j % page
            if codes:
                k, v = (torch.randint(-127, 128, (n, kv, dim), generator=g, dtype=torch.int8) for _ in range(2))
                ks, vs = (torch.rand(n, kv, generator=g) * 0.03 + 0.003 for _ in range(2))
                self.ks[p, :, r], self.vs[p, :, r] = ks, vs
                self.keys.append(k.double() * ks.double()[..., None])
                self.vals.append(v.double() * vs.double()[..., None])
            else:
                k, v = randn(g, n, kv, dim, dtype=dtype), randn(g, n, kv, dim, dtype=dtype)
                self.keys.append(k.double())
                self.vals.append(v.double())
            self.k[p, :, r], self.v[p, :, r] = k, v

    def cache(self):
        dev = lambda t: None if t is None else t.cuda()  # noqa: E731  (keeps the strides)
        return qm.Cache(dev(self.k), dev(self.v), dev(self.ks), dev(self.vs))

    def batch(self, offsets=True, tokens=None):
        news = [new for new, _ in self.seqs]
        off = torch.tensor([0] + list(np.cumsum(news)), dtype=torch.int32).cuda()
        lens = torch.tensor([n for _, n in self.seqs], dtype=torch.int32).cuda()
        return qm.Batch(lens, self.table.cuda(), off if offsets else None, tokens=sum(news) if tokens is None else tokens, max_new=max(news))


def check_attend(paged, q, out, lse, scale, window=0, dtype=None, what=""):
    u = U[dtype or q.dtype]
    at = 0
    group = q.shape[1] // paged.kv
    for i, (new, n) in enumerate(paged.seqs):
        cap = paged.width * paged.page
        want, wl, absv, size = attend_def(q[at: at + new], paged.keys[i], paged.vals[i], new, n, group, scale, window, cap)
        got, gl = out[at: at + new], None if lse is None else lse[at: at + new].double()
        ds = size * (paged.dim + 4) * 2.0 ** -23
        e = (u + 2 * ds[..., None] + 2.0 ** -16) * absv
        fin = torch.isfinite(want)
        assert torch.equal(torch.isnan(got), torch.isnan(want)), (what, i)
        assert torch.equal(got.double()[~fin & ~torch.isnan(want)], want[~fin & ~torch.isnan(want)]), (what, i)
        bad = fin & ~rounded_within(got, want, e)
        assert not bad.any(), (what, i, bad.nonzero()[:4].tolist(), float(((got.double() - want).abs() / e.clamp(min=1e-30))[bad].max()))
        if gl is not None:
            empty = torch.isneginf(wl)
            assert torch.equal(torch.isneginf(gl), empty), (what, i)
            ok = ((gl - wl).abs() <= ds + 2.0 ** -20 * (1 + wl.abs())) | empty | torch.isnan(wl)
            assert ok.all(), (what, i)
        at += new


# ---------------------------------------------------------------- head_norm_rope
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,heads,dim,rot,style", [
    (1, (16, 8), 128, 128, "half"), (3, (5, 1), 64, 32, "pairs"), (37, (7, 3), 80, 80, "half"), (130, (9,), 96, 48, "pairs"),
    (5, (2, 2, 1), 256, 64, "half"), (2, (1,), 8, 8, "half"), (2, (3,), 8, 8, "pairs"), (4097, (16, 8), 128, 128, "half"), (700, (33, 2), 72, 40, "half"),
])
def test_norm_rope(T, heads, dim, rot, style, dtype):
    g = gen(T + dim)
    width = sum(heads) * dim
    rows = randn(g, T, width + 16, dtype=dtype, sigma=3.0)  # heads side by side, and a gap after each token
    table = angles(64, rot)
    pos = torch.randint(0, 64, (T,), generator=g)
    pos[0] = 63
    if T > 2:
        pos[1], pos[2] = -1, 64  # no such rows
    ws = [randn(g, dim, dtype=dtype, sigma=0.3, mean=1.0) for _ in heads]
    if len(ws) > 2:
        ws[1] = None
    d = rows.cuda()
    xs, xd, at = [], [], 0
    for h in heads:
        xs.append(rows[:, at: at + h * dim].unflatten(1, (h, dim)))
        xd.append(d[:, at: at + h * dim].unflatten(1, (h, dim)))
        at += h * dim
    rope = qm.Rope(table.cuda(), style)
    wd = [None if w is None else w.cuda() for w in ws]
    for p in (pos.to(torch.int32), pos):
        got = qm.head_norm_rope(xd, p.cuda(), rope, wd, eps=1e-5)
        for x, w, y in zip(xs, ws, got):
            want, size = norm_rope_def(x, w, 1e-5, table, pos, style)
            assert rounded_within(y.cpu(), want, 2.0 ** -18 * size).all()
    # in place, through the strided views: the same bits, and nothing between them touched
    qm.qm_head_norm_rope(xd, xd, pos.cuda(), rope, wd, 1e-5)
    for x, y in zip(xd, got):
        assert torch.equal(x, y)
    assert torch.equal(d[:, width:].cpu(), rows[:, width:])


def test_norm_rope_norm_only_rope_only_and_specials():
    g = gen(1)
    x = randn(g, 6, 2, 64, dtype=BF)
    x[1, 0] = 0.0
    x[2, 1, 5] = math.inf
    x[3, 0, 7] = math.nan
    w = randn(g, 64, dtype=BF)
    table = angles(8, 64)
    pos = torch.arange(6)
    xd = x.cuda()
    (y,) = qm.head_norm_rope([xd], weights=[w.cuda()], eps=1e-6)
    want, size = norm_rope_def(x, w, 1e-6, None, None, None)
    ok = torch.isfinite(want).all(-1)
    assert rounded_within(y.cpu(), want, 2.0 ** -18 * size)[ok].all()
    assert (y[1, 0] == 0).all() and torch.isnan(y[3, 0]).all() and torch.isnan(y[2, 1, 5]) and (y[2, 1, :5] == 0).all()
    (y,) = qm.head_norm_rope([xd], pos.cuda(), qm.Rope(table.cuda(), "pairs"))
    want, size = norm_rope_def(x, None, 0.0, table, pos, "pairs")
    fin = torch.isfinite(want)
    assert rounded_within(y.cpu(), want, 2.0 ** -18 * size)[fin].all()
    assert not torch.isfinite(y.cpu()[~fin]).any()
    (y,) = qm.head_norm_rope([xd])  # neither: the heads as they are
    nan = torch.isnan(xd)
    assert torch.equal(torch.isnan(y), nan) and torch.equal(y[~nan], xd[~nan])


# ---------------------------------------------------------------- cache_append
APPENDS = [
    # (new, length) of each sequence; heads, dim, rot, page, layout
    ([(1, 1), (1, 0), (1, 77), (1, 16)], 8, 128, 128, 16, "heads"),
    ([(5, 5), (0, 9), (31, 40), (7, 3), (1, 130)], 3, 80, 40, 7, "tokens"),
    ([(300, 301), (1, 2)], 5, 64, 64, 48, "heads"),
    ([(2, 2)], 1, 16, 16, 1, "tokens"),
    ([(4100, 4100)], 2, 96, 96, 256, "heads"),
]


@pytest.mark.parametrize("seqs,kv,dim,rot,page,layout", APPENDS)
@pytest.mark.parametrize("dtype,codes", [(BF, False), (HF, False), (BF, True), (HF, True)])
def test_append(seqs, kv, dim, rot, page, layout, dtype, codes):
    g = gen(len(seqs) + dim)
    P = Paged(g, seqs, kv, dim, page, dtype, codes, layout)
    T = sum(new for new, _ in seqs)
    rows = randn(g, T, 2 * kv * dim, dtype=dtype, sigma=2.0)
    k, v = rows[:, : kv * dim].unflatten(1, (kv, dim)), rows[:, kv * dim:].unflatten(1, (kv, dim))
    w = randn(g, dim, dtype=dtype, sigma=0.2, mean=1.0) if len(seqs) % 2 else None
    style = "half" if page % 2 else "pairs"
    table = angles(max(n for _, n in seqs) + 1, rot)
    cache, batch = P.cache(), P.batch()
    d = rows.cuda()
    kd, vd = d[:, : kv * dim].unflatten(1, (kv, dim)), d[:, kv * dim:].unflatten(1, (kv, dim))
    qm.cache_append(cache, batch, kd, vd, qm.Rope(table.cuda(), style), None if w is None else w.cuda(), 1e-5)
    ck, cv = cache.k.cpu(), cache.v.cpu()
    if codes:
        cks, cvs = cache.k_scales.cpu(), cache.v_scales.cpu()
    wantk, wantv = P.k.clone(), P.v.clone()
    touched = torch.zeros(P.k.shape[:3], dtype=torch.bool)
    at = 0
    for i, (new, n) in enumerate(seqs):
        pos = torch.arange(n - new, n)
        kn, size = norm_rope_def(k[at: at + new], w, 1e-5, table, pos, style)
        for j in range(new):
            p = n - new + j
            if p < 0:
                continue
            page_id, r = int(P.table[i, p // page]), p % page
            touched[page_id, :, r] = True
            for want, sz, got, scales in ((kn[j], size[j], ck, "k"), (v[at + j].double(), None, cv, "v")):
                have = got[page_id, :, r]
                if not codes:
                    assert rounded_within(have, want, 0.0 if sz is None else 2.0 ** -18 * sz).all(), (i, j, scales)
                else:
                    d_ = (cks if scales == "k" else cvs)[page_id, :, r].double()
                    amax = want.abs().amax(-1)
                    assert ((d_ - amax / 127).abs() <= 2.0 ** -17 * amax / 127 + 1e-30).all()
                    assert ((have.double() * d_[:, None] - want).abs() <= d_[:, None] * (0.5 + 127 * 2.0 ** -16)).all()
                    if sz is None:  # the values pass no arithmetic before they are coded: exactly the rule's codes
                        df = (v[at + j].float().abs().amax(-1) / 127.0)
                        inv = torch.where(df == 0, torch.zeros(()), 1.0 / df)
                        x = v[at + j].float() * inv[:, None]
                        q = torch.sign(x) * torch.floor(x.abs() + 0.5)
                        assert torch.equal(have.float(), q)
        at += new
    keep = ~touched
    assert torch.equal(ck[keep].view(torch.uint8), wantk[keep].view(torch.uint8))  # nothing else was written
    assert torch.equal(cv[keep].view(torch.uint8), wantv[keep].view(torch.uint8))


def test_append_specials_of_codes_and_missing_pages():
    g = gen(3)
    P = Paged(g, [(4, 4), (3, 3)], 1, 32, 2, BF, codes=True)
    dropped = int(P.table[1, 1])
    P.table[1, 1] = 10 ** 6  # no such page: position 2 of sequence 1 is dropped
    k = randn(g, 7, 1, 32, dtype=BF)
    k[0, 0, 3] = math.nan
    k[1, 0, 4], k[1, 0, 5] = math.inf, 1.0
    k[2] = 0.0
    cache, batch = P.cache(), P.batch(tokens=7)
    qm.cache_append(cache, batch, k.cuda(), k.cuda())
    s = cache.k_scales.cpu()
    c = cache.k.cpu()
    rows = [(int(P.table[0, p // 2]), p % 2) for p in range(4)]
    assert math.isnan(s[rows[0][0], 0, rows[0][1]]) and (c[rows[0][0], 0, rows[0][1]] == 0).all()
    assert s[rows[1][0], 0, rows[1][1]] == math.inf and (c[rows[1][0], 0, rows[1][1]] == 0).all()
    assert s[rows[2][0], 0, rows[2][1]] == 0 and (c[rows[2][0], 0, rows[2][1]] == 0).all()
    for p, r in rows + [(int(P.table[1, 0]), 0), (int(P.table[1, 0]), 1)]:
        assert torch.equal(cache.v.cpu()[p, :, r], c[p, :, r])
    assert torch.equal(c[dropped], P.k[dropped]) and torch.equal(cache.v.cpu()[dropped], P.v[dropped])


def test_append_rows_of_no_sequence_and_uniform_rows():
    g = gen(4)
    P = Paged(g, [(3, 5), (3, 20), (3, 3)], 2, 64, 4, HF)
    k = randn(g, 9, 2, 64, dtype=HF).cuda()
    v = randn(g, 9, 2, 64, dtype=HF).cuda()
    a, b = P.cache(), P.cache()
    qm.cache_append(a, P.batch(), k, v)
    qm.cache_append(b, P.batch(offsets=False), k, v)
    assert torch.equal(a.k.view(torch.int16), b.k.view(torch.int16)) and torch.equal(a.v.view(torch.int16), b.v.view(torch.int16))
    # two more rows than the sequences have: stored nowhere
    c = P.cache()
    pad = torch.zeros(2, 2, 64, dtype=HF, device="cuda")
    qm.cache_append(c, P.batch(tokens=11), torch.cat([k, pad]), torch.cat([v, pad]))
    assert torch.equal(a.k.view(torch.int16), c.k.view(torch.int16)) and torch.equal(a.v.view(torch.int16), c.v.view(torch.int16))


# ---------------------------------------------------------------- cache_attend
ATTENDS = [
    # (new, length) of each sequence; heads, kv heads, dim, page, window
    ([(1, 1)], 1, 1, 64, 16, 0),
    ([(1, 700)], 16, 8, 128, 16, 0),
    ([(1, 0), (1, 1), (1, 127), (1, 128), (1, 129), (1, 16), (1, 300)], 8, 2, 128, 16, 0),
    ([(1, 1500), (1, 3), (1, 900)], 4, 4, 80, 48, 0),
    ([(1, 257), (1, 258)], 24, 1, 64, 7, 0),
    ([(5, 5), (5, 133), (5, 64)], 14, 2, 64, 32, 0),
    ([(8, 2000), (3, 3), (0, 40), (1, 90)], 10, 2, 96, 300, 0),
    ([(4, 2), (3, 1)], 4, 2, 32, 1, 0),  # more new tokens than the sequence has: the first see nothing
    ([(1, 500), (2, 401), (6, 130)], 6, 3, 128, 16, 100),
    ([(9, 300)], 2, 1, 16, 5, 1),
    ([(7, 140), (1, 133)], 8, 8, 8, 16, 129),
    # chunks
    ([(33, 33)], 2, 1, 128, 16, 0),
    ([(128, 128), (129, 400)], 4, 2, 128, 64, 0),
    ([(300, 555), (1, 1000), (17, 17), (64, 64)], 12, 4, 64, 48, 0),
    ([(200, 900), (0, 0), (1, 5)], 5, 1, 96, 13, 0),
    ([(257, 300), (40, 700)], 8, 8, 112, 32, 65),
    ([(513, 1030)], 7, 1, 128, 128, 0),
    ([(90, 80), (140, 1)], 4, 4, 72, 16, 0),
    ([(600, 640)], 3, 3, 24, 16, 7),
]


@pytest.mark.parametrize("seqs,heads,kv,dim,page,window", ATTENDS)
@pytest.mark.parametrize("dtype,codes", [(BF, False), (HF, False), (BF, True), (HF, True)])
def test_attend(seqs, heads, kv, dim, page, window, dtype, codes):
    if codes and dim % 16:
        pytest.skip("codes come in heads of a multiple of 16")
    g = gen(len(seqs) * 7 + dim + page)
    layout = "tokens" if page % 3 else "heads"
    P = Paged(g, seqs, kv, dim, page, dtype, codes, layout)
    T = sum(new for new, _ in seqs)
    rows = randn(g, T, (heads + 2) * dim, dtype=dtype, sigma=2.0)  # queries within wider rows
    q = rows[:, : heads * dim].unflatten(1, (heads, dim))
    qd = rows.cuda()[:, : heads * dim].unflatten(1, (heads, dim))
    scale = dim ** -0.5
    cache, batch = P.cache(), P.batch()
    out, lse = qm.cache_attend(cache, batch, qd, scale=scale, window=window, lse=True)
    qm.qm_device_status()
    check_attend(P, q, out.cpu(), lse.cpu(), scale, window)
    again = qm.cache_attend(cache, batch, qd, scale=scale, window=window)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))  # the same bits, with or without lse


@pytest.mark.parametrize("new,length,heads,kv", [(1, 9000, 4, 1), (2, 20000, 8, 2), (70, 9000, 2, 1), (300, 6000, 4, 2)])
@pytest.mark.parametrize("codes", [False, True])
def test_attend_split_over_many_ctas(new, length, heads, kv, codes):
    g = gen(length)
    P = Paged(g, [(new, length), (1, 60)], kv, 128, 64, BF, codes)
    q = randn(g, new + 1, heads, 128, dtype=BF, sigma=3.0)
    out, lse = qm.cache_attend(P.cache(), P.batch(), q.cuda(), scale=0.1, lse=True)
    check_attend(P, q, out.cpu(), lse.cpu(), 0.1)


@pytest.mark.parametrize("n,most,heads,kv", [(40, 90, 4, 1), (40, 90, 8, 4), (37, 5, 6, 2), (70, 1, 4, 2)])
@pytest.mark.parametrize("codes", [False, True])
def test_attend_more_sequences_than_a_warp_has_lanes(n, most, heads, kv, codes):
    """An item to each CTA, items kept whole and items split, found past the 32nd sequence, idle ones between."""
    g = gen(n + most + kv)
    seqs = [(0 if i % 9 == 4 else 1 + (i * 37) % most, 100 + (i * 211) % 900) for i in range(n)]
    P = Paged(g, seqs, kv, 64, 16, BF, codes)
    q = randn(g, sum(new for new, _ in seqs), heads, 64, dtype=BF)
    out, lse = qm.cache_attend(P.cache(), P.batch(), q.cuda(), scale=0.125, lse=True)
    qm.qm_device_status()
    check_attend(P, q, out.cpu(), lse.cpu(), 0.125)


@pytest.mark.parametrize("new,length", [(1, 40), (6, 200), (40, 200), (150, 400)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_masked_values_never_reach_a_result(new, length, dtype):
    """A later token's keys and values may be infinite or NaN: earlier tokens' results do not see them."""
    g = gen(new)
    P = Paged(g, [(new, length)], 2, 64, 16, dtype)
    for pos, what in ((length - 1, math.nan), (length - 1 - new // 3, math.inf), (length - 1 - new // 2, -math.inf)):
        r, p = pos % 16, int(P.table[0, pos // 16])
        P.v[p, 0, r, 5] = what
        P.vals[0][pos, 0, 5] = what
        P.v[p, 1, r, :] = what
        P.vals[0][pos, 1, :] = what
    if new > 4:
        pos = length - 2
        P.k[int(P.table[0, pos // 16]), 0, pos % 16, 3] = math.nan
        P.keys[0][pos, 0, 3] = math.nan
    q = randn(g, new, 4, 64, dtype=dtype)
    out = qm.cache_attend(P.cache(), P.batch(), q.cuda(), scale=0.125)
    want = attend_def(q, P.keys[0], P.vals[0], new, length, 2, 0.125, 0, 1 << 30)[0]
    assert torch.isfinite(want[: max(1, new - 1 - new // 2) if new > 1 else 0]).all()
    check_attend(P, q, out.cpu(), None, 0.125)


def test_masked_scales_never_reach_a_result():
    g = gen(9)
    P = Paged(g, [(20, 90), (3, 30)], 2, 64, 16, BF, codes=True)
    for pos, what in ((89, math.nan), (80, math.inf)):
        p, r = int(P.table[0, pos // 16]), pos % 16
        P.vs[p, 0, r] = what
        P.vals[0][pos, 0] = P.v[p, 0, r].double() * what
        P.ks[p, 1, r] = math.nan
        P.keys[0][pos, 1] = math.nan
    q = randn(g, 23, 4, 64, dtype=BF)
    out = qm.cache_attend(P.cache(), P.batch(), q.cuda(), scale=0.125)
    check_attend(P, q, out.cpu(), None, 0.125)


@pytest.mark.parametrize("new", [1, 4, 70])
@pytest.mark.parametrize("codes", [False, True])
def test_missing_pages_read_as_zeros(new, codes):
    g = gen(11)
    P = Paged(g, [(new, 300)], 2, 64, 16, HF, codes)
    for page, bad in ((0, -1), (7, -5), (11, 1 << 30)):
        P.table[0, page] = bad
        P.keys[0][page * 16: page * 16 + 16] = 0
        P.vals[0][page * 16: page * 16 + 16] = 0
    q = randn(g, new, 4, 64, dtype=HF)
    out, lse = qm.cache_attend(P.cache(), P.batch(), q.cuda(), scale=0.2, lse=True)
    check_attend(P, q, out.cpu(), lse.cpu(), 0.2)


@pytest.mark.parametrize("new", [1, 50])
def test_length_past_the_page_table_is_cut(new):
    g = gen(12)
    P = Paged(g, [(new, 160)], 1, 64, 16, BF, spare=0)
    batch = P.batch()
    batch.lens += 33  # the table has room for 160
    q = randn(g, new, 2, 64, dtype=BF)
    out, lse = qm.cache_attend(P.cache(), batch, q.cuda(), scale=0.125, lse=True)
    P.seqs = [(new, 193)]
    check_attend(P, q, out.cpu(), lse.cpu(), 0.125)


@pytest.mark.parametrize("new", [1, 40])
def test_large_and_infinite_scores(new):
    g = gen(13)
    P = Paged(g, [(new, 260)], 1, 64, 16, BF)
    q = randn(g, new, 2, 64, dtype=BF, sigma=40.0)
    pos = 100
    p, r = int(P.table[0, pos // 16]), pos % 16
    # every score of query head 1 falls to -inf: q >= 0 against keys that hold -inf in one element
    q[:, 1, :] = 1.0
    P.k[:, 0, :, 0] = torch.where(torch.isnan(P.k[:, 0, :, 0]), P.k[:, 0, :, 0], torch.full_like(P.k[:, 0, :, 0], -math.inf))
    P.keys[0][:, 0, 0] = -math.inf
    q[:, 0, 0] = 0.0  # 0 * -inf: NaN for head 0
    out, lse = qm.cache_attend(P.cache(), P.batch(), q.cuda(), scale=1.0, lse=True)
    assert torch.isnan(out).all()
    assert torch.isnan(lse[:, 0]).all() and torch.isneginf(lse[:, 1]).all()
    P = Paged(g, [(new, 260)], 1, 64, 16, BF)
    q = randn(g, new, 2, 64, dtype=BF, sigma=40.0)
    out, lse = qm.cache_attend(P.cache(), P.batch(), q.cuda(), scale=1.0, lse=True)
    check_attend(P, q, out.cpu(), lse.cpu(), 1.0)


@pytest.mark.parametrize("new,heads,dim", [(1, 4, 128), (5, 8, 128), (9, 8, 64), (3, 4, 96), (70, 8, 128)])
@pytest.mark.parametrize("e", [-100, -60, 14, 60, 96])
def test_queries_of_any_size_over_codes(new, heads, dim, e):
    """Rows from 2^(e-12) to 2^e, one with an element 2^12 above the rest: a power of two is exact
    throughout, so the bits are those of e = 0, and the scores' log-sum-exp keeps its bound."""
    g = gen(31)
    P = Paged(g, [(new, 300), (1, 20)], 1, dim, 32, BF, True)
    q = (randn(g, new + 1, heads, dim, sigma=16.0).round() / 16).clamp(-3.5, 3.5)
    q *= 2.0 ** -(torch.arange(heads) % 5 * 3.0)[None, :, None]
    q[:, 1, 3] *= 2.0 ** 12
    q = q.to(BF)
    cache, batch = P.cache(), P.batch()
    got, want = (qm.cache_attend(cache, batch, (q.double() * 2.0 ** x).to(BF).cuda(), scale=2.0 ** -x / 8, lse=True) for x in (e, 0))
    qm.qm_device_status()
    assert torch.equal(got[0].view(torch.int16), want[0].view(torch.int16))
    assert torch.equal(got[1].view(torch.int32), want[1].view(torch.int32))
    at, lse = 0, want[1].cpu().double()
    for i, (n, length) in enumerate(P.seqs):
        _, wl, _, size = attend_def(q[at: at + n], P.keys[i], P.vals[i], n, length, heads, 0.125, 0, P.width * P.page)
        ds = size * (dim + 4) * 2.0 ** -23
        assert ((lse[at: at + n] - wl).abs() <= ds + 2.0 ** -20 * (1 + wl.abs())).all()
        at += n


@pytest.mark.parametrize("new", [1, 5, 40])
def test_infinite_queries_over_codes(new):
    g = gen(29)
    P = Paged(g, [(new, 260)], 1, 64, 16, BF, True)
    P.k[..., 0] = P.k[..., 0].abs().clamp(min=1)  # the infinity meets codes above zero alone
    q = randn(g, new, 3, 64, dtype=BF)
    q[:, 0, 0] = -math.inf  # every score -inf, whatever the rest of the row holds
    q[:, 0, 1:] = q[:, 0, 1:].sign() * 2.0 ** 100
    q[:, 1, 0] = math.nan
    out, lse = qm.cache_attend(P.cache(), P.batch(), q.cuda(), scale=1.0, lse=True)
    assert torch.isneginf(lse[:, 0]).all() and torch.isnan(out[:, 0]).all()
    assert torch.isnan(lse[:, 1]).all() and torch.isnan(out[:, 1]).all()
    assert torch.isfinite(out[:, 2]).all() and torch.isfinite(lse[:, 2]).all()


def test_rows_of_no_sequence_are_not_written():
    g = gen(14)
    P = Paged(g, [(3, 50), (40, 60)], 2, 64, 16, BF)
    q = randn(g, 48, 4, 64, dtype=BF)
    batch = P.batch(tokens=48)
    out = torch.full((48, 4, 64), 7.0, dtype=BF, device="cuda")
    cache = P.cache()
    ws = torch.empty(qm.qm_cache_attend_workspace(cache, batch, 4), dtype=torch.uint8, device="cuda")
    qm.qm_cache_attend(cache, batch, q.cuda(), out, 0.125, ws)
    assert (out[43:] == 7).all()
    check_attend(P, q, out[:43].cpu(), None, 0.125)


@pytest.mark.parametrize("codes", [True, False])
def test_offsets_past_32_bits(codes):
    """A cache of more than 2^31 elements a part, used at both of its ends."""
    g = gen(15)
    kv, page, dim = 2, 128, 128
    pages = (1 << 31) // (kv * page * dim) + 40
    k = torch.empty(pages, kv, page, dim, dtype=torch.int8 if codes else BF, device="cuda")
    v = torch.empty_like(k)
    ks, vs = (torch.full((pages, kv, page), math.nan, device="cuda") if codes else None for _ in range(2))
    ids = [pages - 1, 0, pages - 30, 5]
    seqs = [(1, 400), (60, 100)]
    table = torch.tensor([ids, [pages - 2, -1, -1, -1]], dtype=torch.int32)
    small = Paged(g, seqs, kv, dim, page, BF, codes=codes)
    for i in range(2):
        for j in range(-(-seqs[i][1] // page)):
            src, dst = int(small.table[i, j]), int(table[i, j])
            k[dst], v[dst] = small.k[src].cuda(), small.v[src].cuda()
            if codes:
                ks[dst], vs[dst] = small.ks[src].cuda(), small.vs[src].cuda()
    cache = qm.Cache(k, v, ks, vs)
    off = torch.tensor([0, 1, 61], dtype=torch.int32).cuda()
    lens = torch.tensor([400, 100], dtype=torch.int32).cuda()
    q = randn(g, 61, 4, dim, dtype=BF)
    for most in (60, 1):  # either kernel
        batch = qm.Batch(lens, table.cuda(), off, tokens=61, max_new=most)
        out = qm.cache_attend(cache, batch, q.cuda(), scale=0.1)
        check_attend(small, q, out.cpu(), None, 0.1)
    new = randn(g, 61, kv, dim, dtype=BF)
    qm.cache_append(cache, batch, new.cuda(), new.cuda())
    for p, r, i in ((5, 399 - 3 * page, 0), (pages - 2, 99, 60)):
        got = cache.v[p, :, r].cpu().double()
        if codes:
            got = got * cache.v_scales[p, :, r].cpu().double()[:, None]
        assert (got - new[i].double()).abs().max() < (0.05 if codes else 1e-30)


def test_another_stream_and_a_captured_graph():
    g = gen(16)
    P = Paged(g, [(1, 300), (1, 40), (1, 999)], 2, 128, 16, BF)
    kv, heads, dim = 2, 4, 128
    rows = randn(g, 3, (heads + 2 * kv) * dim, dtype=BF)
    table = angles(1000, dim).cuda()
    cache, batch, rope = P.cache(), P.batch(), qm.Rope(table)
    x = rows.cuda()
    q, k, v = (x[:, a * dim: b * dim].unflatten(1, (b - a, dim)) for a, b in ((0, heads), (heads, heads + kv), (heads + kv, heads + 2 * kv)))
    pos = torch.tensor([299, 39, 998], dtype=torch.int32).cuda()
    ws = torch.empty(qm.qm_cache_attend_workspace(cache, batch, heads), dtype=torch.uint8, device="cuda")
    qr, out = torch.empty(3, heads, dim, dtype=BF, device="cuda"), torch.empty(3, heads, dim, dtype=BF, device="cuda")

    def step(stream=None):
        qm.qm_head_norm_rope([q], [qr], pos, rope, stream=stream)
        qm.qm_cache_append(cache, batch, k, v, rope, stream=stream)
        qm.qm_cache_attend(cache, batch, qr, out, dim ** -0.5, ws, stream=stream)

    step()
    want = out.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out.zero_()
    torch.cuda.synchronize()
    step(s)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    # the step against the definition
    kk, _ = norm_rope_def(rows[:, heads * dim: (heads + kv) * dim].unflatten(1, (kv, dim)), None, 0, table.cpu(), pos.cpu(), "half")
    for i, (_, n) in enumerate(P.seqs):
        P.keys[i][n - 1] = kk[i].to(BF).double()
        P.vals[i][n - 1] = rows[i, (heads + kv) * dim:].unflatten(0, (kv, dim)).double()
    check_attend(P, qr.cpu(), out.cpu(), None, dim ** -0.5)


def test_nothing_to_do():
    P = Paged(gen(17), [(1, 4)], 1, 64, 16, BF)
    cache = P.cache()
    empty = torch.empty(0, 2, 64, dtype=BF, device="cuda")
    batch = qm.Batch(torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, 1, dtype=torch.int32, device="cuda"))
    assert qm.cache_attend(cache, batch, empty).shape == (0, 2, 64)
    qm.cache_append(cache, batch, empty[:, :1], empty[:, :1])
    (y,) = qm.head_norm_rope([empty])
    assert y.shape == (0, 2, 64)
    # sequences without new tokens: no rows, nothing read
    batch = qm.Batch(P.batch().lens, P.table.cuda(), torch.zeros(2, dtype=torch.int32, device="cuda"), tokens=0)
    assert qm.cache_attend(cache, batch, empty).shape == (0, 2, 64)
    # and a batch whose rows belong to no sequence
    batch = qm.Batch(P.batch().lens, P.table.cuda(), torch.zeros(2, dtype=torch.int32, device="cuda"), tokens=3)
    out = qm.cache_attend(cache, batch, torch.zeros(3, 2, 64, dtype=BF, device="cuda"))
    assert out.shape == (3, 2, 64)
    qm.qm_device_status()


def test_norm_rope_more_tokens_than_one_launch_takes():
    T = 65535 * 16 + 37  # heads of 64 elements or fewer: 16 tokens to a block
    g = gen(20)
    x = randn(g, T, 1, 8, dtype=BF)
    w = randn(g, 8, dtype=BF)
    table = angles(32, 8)
    pos = torch.arange(T) % 32
    (y,) = qm.head_norm_rope([x.cuda()], pos.cuda(), qm.Rope(table.cuda()), [w.cuda()])
    want, size = norm_rope_def(x, w, 1e-6, table, pos, "half")
    assert rounded_within(y.cpu(), want, 2.0 ** -18 * size).all()


def test_calls_on_a_side_stream_own_their_tensors():
    g = gen(21)
    P = Paged(g, [(1, 5000), (1, 700)], 2, 128, 16, BF)
    q = randn(g, 2, 4, 128, dtype=BF).cuda()
    cache, batch = P.cache(), P.batch()
    s = torch.cuda.Stream()
    want = qm.cache_attend(cache, batch, q)
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        got = []
        for _ in range(20):
            got.append(qm.cache_attend(cache, batch, q, stream=stream))
            torch.full((1 << 20,), 7, dtype=torch.int32, device="cuda")  # would take the workspace's memory, were it this stream's
        torch.cuda.synchronize()
        for o in got:
            assert torch.equal(o, want)


def test_strides_of_axes_of_one_do_not_count():
    g = gen(22)
    P = Paged(g, [(1, 90)], 1, 64, 16, BF)
    q = randn(g, 1, 1, 64, dtype=BF)
    odd = q.cuda().as_strided((1, 1, 64), (3, 5, 1))
    out = qm.cache_attend(P.cache(), P.batch(), odd, scale=0.125)
    check_attend(P, q, out.cpu(), None, 0.125)
    (a,) = qm.head_norm_rope([odd], weights=[torch.ones(64, dtype=BF, device="cuda")])
    (b,) = qm.head_norm_rope([q.cuda()], weights=[torch.ones(64, dtype=BF, device="cuda")])
    assert torch.equal(a, b)


def test_no_part_flag_stays_set():
    """Items split between CTAs leave the workspace's flags (its first eight bytes a CTA) as a replay has to find them."""
    g = gen(51)
    P = Paged(g, [(1, 5000), (1, 700), (1, 3000)], 2, 128, 16, BF)
    q = randn(g, 3, 4, 128, dtype=BF)
    cache, batch = P.cache(), P.batch()
    ws = torch.zeros(qm.qm_cache_attend_workspace(cache, batch, 4), dtype=torch.uint8, device="cuda")
    flags = ws[: 8 * torch.cuda.get_device_properties(0).multi_processor_count]
    for _ in range(3):
        out = qm.cache_attend(cache, batch, q.cuda(), scale=0.1, workspace=ws)
        assert not flags.any() and ws.any()
        check_attend(P, q, out.cpu(), None, 0.1)


def far_codes(g, seqs, kv, dim, page, kind):
    """A cache of codes, none of them 0, with value scales of either sign and of any size."""
    P = Paged(g, seqs, kv, dim, page, BF, codes=True)
    for i, (_, n) in enumerate(seqs):
        j = torch.arange(n)
        p, r = P.table[i].long()[j // page], j % page
        v = torch.randint(1, 128, (n, kv, dim), generator=g) * (torch.randint(0, 2, (n, kv, dim), generator=g) * 2 - 1)
        vs = (torch.rand(n, kv, generator=g) * 0.03 + 0.003) * (torch.randint(0, 2, (n, kv), generator=g) * 2 - 1)
        if kind == "any":
            vs = vs.double() * 2.0 ** torch.randint(-110, 111, (n, kv), generator=g).double()
        else:
            vs = vs.double() * 2.0 ** kind
        vs[torch.rand(n, kv, generator=g) < 0.05] = 0.0
        P.v[p, :, r], P.vs[p, :, r] = v.to(torch.int8), vs.float()
        P.vals[i] = v.double() * vs.float().double()[..., None]
    return P


@pytest.mark.parametrize("kind", [0, -115, -85, -78, -40, 40, 78, 85, 110, "any"])
@pytest.mark.parametrize("new,length,heads,dim", [(1, 700, 4, 128), (5, 300, 8, 64), (5, 300, 6, 96), (70, 400, 4, 128), (200, 300, 2, 80), (1, 9000, 3, 128)])
def test_value_scales_of_any_size_and_sign(new, length, heads, dim, kind):
    """A code's scale is any finite float32: nothing overflows or vanishes on its way to a bfloat16 result."""
    g = gen(41)
    P = far_codes(g, [(new, length), (1, 40)], 1, dim, 16, kind)
    q = randn(g, new + 1, heads, dim, dtype=BF)
    out, lse = qm.cache_attend(P.cache(), P.batch(), q.cuda(), scale=dim ** -0.5, lse=True)
    qm.qm_device_status()
    check_attend(P, q, out.cpu(), None, dim ** -0.5)
    # the total is held against a maximum that counts the scales: the logarithm is a difference of two numbers of up to
    # 80 more each in powers of two, rounded in float32
    at = 0
    for i, (n, length_) in enumerate(P.seqs):
        _, wl, _, size = attend_def(q[at: at + n], P.keys[i], P.vals[i], n, length_, heads, dim ** -0.5, 0, P.width * P.page)
        ds = size * (dim + 4) * 2.0 ** -23
        assert ((lse[at: at + n].cpu() - wl).abs() <= ds + 2.0 ** -20 * (1 + wl.abs() + 80)).all()
        at += n


@pytest.mark.parametrize("new", [1, 5, 70])
def test_negative_value_scales_in_float16(new):
    g = gen(43)
    P = far_codes(g, [(new, 300)], 2, 64, 32, 0)
    q = randn(g, new, 4, 64, dtype=HF)
    out, lse = qm.cache_attend(P.cache(), P.batch(), q.cuda(), scale=0.125, lse=True)
    check_attend(P, q, out.cpu(), lse.cpu(), 0.125)


@pytest.mark.parametrize("new,length", [(1, 200), (1, 9000), (5, 300), (60, 400), (300, 3000)])
@pytest.mark.parametrize("dtype,codes", [(BF, False), (HF, False), (BF, True), (HF, True)])
def test_a_score_of_infinity(new, length, dtype, codes):
    """The log-sum-exp of a row with a score of +infinity is +infinity, of one with a NaN among its scores NaN; the weights are
    the definition's infinity less infinity either way."""
    g = gen(47)
    P = Paged(g, [(new, length), (2, 50)], 1, 64, 16, dtype, codes)

    def put(pos, what):  # the key at a position of sequence 0 (codes: its scale), and the definition's
        p, r = int(P.table[0, pos // 16]), pos % 16
        if codes:
            P.k[p, 0, r] = P.k[p, 0, r].abs().clamp(min=1)
            P.ks[p, 0, r] = what
            P.keys[0][pos, 0] = P.k[p, 0, r].double() * what
        else:
            P.k[p, 0, r, 7] = what
            P.keys[0][pos, 0, 7] = what

    put(length // 3, math.inf)
    put(length // 3 + 5, -math.inf)
    if new > 4:
        put(length - 2, math.nan)  # the last two tokens see this one too
    q = randn(g, new + 2, 3, 64, dtype=dtype).abs()  # so that an infinity's sign is its score's
    q[:, 2] = -q[:, 2]
    out, lse = qm.cache_attend(P.cache(), P.batch(), q.cuda(), scale=0.125, lse=True)
    qm.qm_device_status()
    out, lse = out.cpu(), lse.cpu()
    seen = new - 2 if new > 4 else new  # rows that see no NaN
    if new <= length - length // 3 - 6:  # every row sees both infinities
        assert torch.isposinf(lse[:seen]).all()
        assert torch.isnan(out[:new]).all() and torch.isnan(lse[seen:new]).all()
    assert torch.isfinite(lse[new:]).all()
    check_attend(P, q, out, None, 0.125)


@pytest.mark.parametrize("news", [
    # new tokens of each sequence by replay; the rows of a call stay as many
    [(1, 1, 1, 1)] * 6,                                                             # few rows to a key head
    [(40, 300, 0, 100), (440, 0, 0, 0), (110, 110, 110, 110), (0, 0, 439, 1), (40, 300, 0, 100), (1, 1, 437, 1)],  # chunks, joined after
    [(3, 5, 0, 4), (5, 5, 2, 0), (0, 0, 12, 0), (3, 5, 0, 4), (1, 1, 1, 9), (12, 0, 0, 0)],
])
@pytest.mark.parametrize("codes", [False, True])
def test_a_captured_call_replayed_over_other_lengths(news, codes):
    """Lengths, rows and page table change in place between replays: items are split, whole and gone again, and
    each replay gives the bits of a plain call."""
    g = gen(53)
    T, kv, heads, dim, page = sum(news[0]), 2, 4, 128, 16
    P = Paged(g, [(0, 4000)] * 4, kv, dim, page, BF, codes)
    lengths = [(4000, 10, 3, 700), (0, 4000, 4000, 0), (900, 901, 902, 903), (64, 0, 3999, 5), (4000, 10, 3, 700), (1, 1, 2500, 1)]
    q = randn(g, T, heads, dim, dtype=BF).cuda()
    cache, i32 = P.cache(), dict(dtype=torch.int32, device="cuda")
    lens, table, offsets = torch.zeros(4, **i32), P.table.cuda(), torch.zeros(5, **i32)
    batch = qm.Batch(lens, table, offsets, tokens=T, max_new=max(max(n) for n in news))
    ws = torch.empty(qm.qm_cache_attend_workspace(cache, batch, heads), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty(T, heads, dim, dtype=BF, device="cuda"), torch.empty(T, heads, device="cuda")

    def put(i):
        lens.copy_(torch.tensor([max(n, m) for n, m in zip(lengths[i], news[i])], **i32))
        offsets.copy_(torch.tensor([0] + list(np.cumsum(news[i])), **i32))
        table.copy_(P.table.roll(i, 0))

    def call(to, total):
        qm.qm_cache_attend(cache, batch, q, to, 0.1, ws, lse=total)

    put(0)
    call(out, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, lse)
    for i in list(range(len(news))) * 2:
        put(i)
        for _ in range(3):
            out.zero_()
            lse.zero_()
            graph.replay()
        want, total = torch.zeros_like(out), torch.zeros_like(lse)
        call(want, total)
        qm.qm_device_status()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(lse.view(torch.int32), total.view(torch.int32)), i
    put(2)  # and the definition's values
    graph.replay()
    P.seqs = list(zip(news[2], lens.tolist()))
    P.keys, P.vals = (x[-2:] + x[:-2] for x in (P.keys, P.vals))
    check_attend(P, q.cpu(), out.cpu(), lse.cpu(), 0.1)
