"""The cache operators' refusals, on the host: every case fails validation
before any CUDA call and names the part."""
import ctypes
import math

import pytest
import torch

import packed_qmatmul_gb300 as qm

A = 4096  # an aligned address nothing reads


@pytest.fixture(scope="module")
def lib():
    from packed_qmatmul_gb300 import build

    build.build()
    return qm.load_library()


def heads(data=A, ts=1024, hs=64, n=2, dt=qm.QM_BF16):
    return qm._HEADS(data, ts, hs, n, dt)


def rope(table=A, rows=10, dim=64, style=qm.QM_ROPE_HALF):
    return qm._ROPE(table, rows, dim, style)


def cache(k=A, v=A, ks=0, vs=0, ps=2048, hs=1024, ts=64, sps=0, shs=0, sts=0, pages=4, dt=qm.QM_BF16, n=2, dim=64, page=16):
    return qm._CACHE(k, v, ks, vs, ps, hs, ts, sps, shs, sts, pages, dt, n, dim, page)


def batch(lens=A, table=A, off=A, tokens=3, width=5, stride=5, seqs=2, max_new=0):
    return qm._BATCH(lens, table, off, tokens, width, stride, seqs, max_new)


def refused(lib, st, part, status=qm.QM_EINVAL):
    msg = lib.qm_last_error().decode()
    assert st == status and msg.startswith(part), (st, msg)


def test_struct_sizes():
    assert [len(x) for x in (heads(), rope(), cache(), batch())] == [32, 24, 104, 56]


@pytest.mark.parametrize("part,change", [
    ("count", dict(count=0)), ("count", dict(count=5)), ("x", dict(xs=None)), ("out", dict(outs=None)), ("x", dict(T=-1)), ("x", dict(T=1 << 31)),
    ("x", dict(dim=60)), ("x", dict(dim=0)), ("eps", dict(eps=-1.0)), ("eps", dict(eps=math.nan)), ("eps", dict(eps=math.inf)),
    ("x[0]", dict(xs=heads(data=0))), ("x[0]", dict(xs=heads(data=A + 8))), ("x[0]", dict(xs=heads(ts=1028))), ("x[0]", dict(xs=heads(hs=-64))),
    ("x[0]", dict(xs=heads(n=0))), ("x[0]", dict(xs=heads(dt=qm.QM_F32))), ("out[0]", dict(outs=heads(dt=qm.QM_F16))),
    ("out[0]", dict(outs=heads(n=3))), ("out[0]", dict(outs=heads(hs=32))), ("out[0]", dict(outs=heads(ts=0))), ("out[0]", dict(outs=heads(ts=2048))),
    ("weights[0]", dict(weights=A + 2)), ("rope", dict(rope=rope(style=2))), ("rope", dict(rope=rope(dim=72))), ("rope", dict(rope=rope(dim=12))),
    ("rope", dict(rope=rope(table=0))), ("rope", dict(rope=rope(table=A + 4))), ("rope", dict(rope=rope(rows=-1))),
    ("positions", dict(pos=0)), ("positions", dict(pos=A + 2)), ("positions", dict(ptype=7)),
])
def test_norm_rope_refusals(lib, part, change):
    a = dict(xs=heads(), outs=heads(), weights=0, count=1, T=3, dim=64, eps=1e-6, rope=rope(), pos=A, ptype=qm.QM_I32) | change
    w = (ctypes.c_void_p * 1)(a["weights"])
    refused(lib, lib.qm_head_norm_rope(a["xs"], a["outs"], w, a["count"], a["T"], a["dim"], a["eps"], a["rope"], a["pos"], a["ptype"], None), part)


def test_norm_rope_widest_head(lib):
    st = lib.qm_head_norm_rope(heads(hs=264), heads(hs=264), None, 1, 3, 264, 0.0, None, None, qm.QM_I32, None)
    refused(lib, st, "x", qm.QM_ENOTSUP)


CACHE = [
    ("cache", None), ("cache", dict(dt=qm.QM_F32)), ("cache", dict(dim=60)), ("cache", dict(dim=0)), ("cache", dict(n=0)), ("cache", dict(page=0)),
    ("cache", dict(pages=-1)), ("cache", dict(ps=2052)), ("cache", dict(hs=-1024)), ("cache", dict(ts=32)), ("cache", dict(ps=0)),
    ("k", dict(k=0)), ("v", dict(v=0)), ("k", dict(k=A + 8)), ("v", dict(v=A + 2)), ("k_scales", dict(ks=A)), ("v_scales", dict(vs=A)),
    ("k_scales", dict(dt=qm.QM_I8)), ("v_scales", dict(dt=qm.QM_I8, ks=A)), ("k_scales", dict(dt=qm.QM_I8, ks=A + 2, vs=A)),
    ("k_scales", dict(dt=qm.QM_I8, ks=A, vs=A, sts=-1)), ("cache", dict(dt=qm.QM_I8, ks=A, vs=A, dim=72)),
]
BATCH = [
    ("batch", None), ("batch", dict(seqs=-1)), ("batch", dict(tokens=-1)), ("batch", dict(tokens=1 << 31)), ("batch", dict(max_new=-1)),
    ("page_table", dict(width=-1)), ("page_table", dict(stride=-1)), ("q_offsets", dict(off=0)), ("lens", dict(lens=0)), ("lens", dict(lens=A + 1)),
    ("page_table", dict(table=0)), ("page_table", dict(table=A + 2)), ("q_offsets", dict(off=A + 2)),
]


@pytest.mark.parametrize("part,c,b", [(p, c, {}) for p, c in CACHE] + [(p, {}, b) for p, b in BATCH])
def test_cache_and_batch_refusals(lib, part, c, b):
    c, b = (None if x is None else f(**x) for f, x in ((cache, c), (batch, b)))
    refused(lib, lib.qm_cache_append(c, b, heads(), heads(), None, 0.0, None, None), part)
    refused(lib, lib.qm_cache_attend(c, b, heads(), heads(data=8192), None, 1.0, 0, A, 1 << 40, None), part)
    assert lib.qm_cache_attend_workspace(c, b, 2) == 0


@pytest.mark.parametrize("part,change", [
    ("k", dict(k=heads(n=3))), ("v", dict(v=heads(n=1))), ("v", dict(v=heads(dt=qm.QM_F16))), ("k", dict(k=heads(dt=qm.QM_F16), v=heads(dt=qm.QM_F16))),
    ("k", dict(k=None)), ("v", dict(v=heads(data=0))), ("k_weight", dict(w=A + 4)), ("eps", dict(eps=-1.0)), ("rope", dict(rope=rope(dim=128))),
])
def test_append_refusals(lib, part, change):
    a = dict(k=heads(), v=heads(), w=None, eps=0.0, rope=rope()) | change
    refused(lib, lib.qm_cache_append(cache(), batch(), a["k"], a["v"], a["w"], a["eps"], a["rope"], None), part)


@pytest.mark.parametrize("part,change", [
    ("q", dict(q=heads(n=3))), ("q", dict(q=heads(dt=qm.QM_F16))), ("q", dict(q=heads(data=A + 8))), ("q", dict(q=None)), ("out", dict(out=None)),
    ("out", dict(out=heads(data=8192, n=4))), ("out", dict(out=heads(data=8192, dt=qm.QM_F16))), ("out", dict(out=heads(data=A))),
    ("out", dict(out=heads(data=8192, ts=32))), ("lse", dict(lse=A + 2)), ("scale", dict(scale=0.0)), ("scale", dict(scale=-1.0)),
    ("scale", dict(scale=math.nan)), ("window", dict(window=-1)), ("workspace", dict(ws=0)), ("workspace", dict(size=64)), ("workspace", dict(ws=A + 8)),
    ("workspace", dict(ws=A + 16)),
])
def test_attend_refusals(lib, part, change):
    a = dict(q=heads(), out=heads(data=8192), lse=None, scale=1.0, window=0, ws=A, size=1 << 40) | change
    refused(lib, lib.qm_cache_attend(cache(), batch(), a["q"], a["out"], a["lse"], a["scale"], a["window"], a["ws"], a["size"], None), part)


def test_wide_heads_are_not_supported(lib):
    c = cache(dim=136, ts=136, hs=136 * 16, ps=136 * 32)
    refused(lib, lib.qm_cache_append(c, batch(), heads(), heads(), None, 0.0, None, None), "cache", qm.QM_ENOTSUP)


def test_workspace_size_depends_on_shapes(lib):
    assert lib.qm_cache_attend_workspace(cache(), batch(), 2) % 256 == 0
    assert lib.qm_cache_attend_workspace(cache(), batch(), 2) > 0
    assert lib.qm_cache_attend_workspace(cache(), batch(), 3) == 0
    assert lib.qm_cache_attend_workspace(cache(), batch(tokens=0), 2) == 0


def test_binding_refusals():
    k = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    lens, table = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32)
    c, b = qm.Cache(k, k), qm.Batch(lens, table)
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    for f in (
        lambda: qm.Cache(k, k[:2]), lambda: qm.Cache(k, k.half()), lambda: qm.Cache(k.float(), k.float()), lambda: qm.Cache(k, k.permute(0, 2, 1, 3)),
        lambda: qm.Cache(k.transpose(2, 3), k.transpose(2, 3)), lambda: qm.Cache(k, k, torch.zeros(3, 2, 16), torch.zeros(3, 2, 16)),
        lambda: qm.Cache(k.to(torch.int8), k.to(torch.int8)), lambda: qm.Cache(k.to(torch.int8), k.to(torch.int8), torch.zeros(3, 2), torch.zeros(3, 2)),
        lambda: qm.Batch(lens.long(), table), lambda: qm.Batch(lens, table[:1]), lambda: qm.Batch(lens, table.long()), lambda: qm.Batch(lens, table, lens),
        lambda: qm.Rope(torch.zeros(3, 64).double()), lambda: qm.Rope(torch.zeros(3, 64), "other"),
        lambda: qm.cache_append(c, b, x[:1], x), lambda: qm.cache_append(c, b, x, x[..., :32]), lambda: qm.cache_append(c, b, x.transpose(1, 2), x),
        lambda: qm.cache_append(c, b, x, x, k_weight=torch.zeros(32, dtype=torch.bfloat16)),
        lambda: qm.head_norm_rope([]), lambda: qm.head_norm_rope([x] * 5), lambda: qm.head_norm_rope([x, x[:1]]),
        lambda: qm.head_norm_rope([x], weights=[torch.zeros(32, dtype=torch.bfloat16)]), lambda: qm.head_norm_rope([x], torch.zeros(3, dtype=torch.int32)),
        lambda: qm.head_norm_rope([x], torch.zeros(2)), lambda: qm.qm_cache_attend(c, b, x[:1], x, 1.0, None),
        lambda: qm.qm_cache_attend(c, b, x, x, 1.0, None, lse=torch.zeros(2, 3)),
    ):
        with pytest.raises(qm.QMError) as e:
            f()
        assert e.value.status == qm.QM_EINVAL


class Elsewhere:
    """A tensor that says it is on another device."""

    def __init__(self, t, gpu):
        self.t, self.gpu = t, gpu

    def get_device(self):
        return self.gpu

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.mark.parametrize("gpu,why", [(-1, "not on a GPU"), (1, "on another GPU than")])
def test_every_tensor_of_a_call_is_on_one_gpu(gpu, why):
    """A tensor of the host, or of another GPU, is refused by name before the library is called."""
    def on(t, here=0):
        return Elsewhere(t, here)

    bf = torch.bfloat16
    x, w = torch.zeros(2, 2, 64, dtype=bf), torch.zeros(64, dtype=bf)
    k, lens, table = torch.zeros(3, 2, 16, 64, dtype=bf), torch.zeros(2, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32)
    ws, lse, pos, turns = torch.zeros(8, dtype=torch.uint8), torch.zeros(2, 2), torch.zeros(2, dtype=torch.int32), torch.zeros(4, 64)

    def cache(at=0):
        return qm.Cache(on(k, at), on(k, at))

    def batch(at=0):
        return qm.Batch(on(lens, at), on(table, at))

    def rope(at=0):
        return qm.Rope(on(turns, at))

    calls = [
        ("x", lambda: qm.qm_head_norm_rope([on(x), on(x, gpu)], [on(x), on(x)])), ("out", lambda: qm.qm_head_norm_rope([on(x)], [on(x, gpu)])),
        ("weights", lambda: qm.qm_head_norm_rope([on(x), on(x)], [on(x), on(x)], weights=[None, on(w, gpu)])),
        ("positions", lambda: qm.qm_head_norm_rope([on(x)], [on(x)], on(pos, gpu), rope())),
        ("rope", lambda: qm.qm_head_norm_rope([on(x)], [on(x)], on(pos), rope(gpu))),
        ("batch", lambda: qm.cache_append(cache(), batch(gpu), on(x), on(x))), ("k", lambda: qm.cache_append(cache(), batch(), on(x, gpu), on(x))),
        ("v", lambda: qm.cache_append(cache(), batch(), on(x), on(x, gpu))), ("rope", lambda: qm.cache_append(cache(), batch(), on(x), on(x), rope(gpu))),
        ("k_weight", lambda: qm.cache_append(cache(), batch(), on(x), on(x), rope(), on(w, gpu))),
        ("batch", lambda: qm.qm_cache_attend(cache(), batch(gpu), on(x), on(x), 1.0, on(ws))),
        ("q", lambda: qm.qm_cache_attend(cache(), batch(), on(x, gpu), on(x), 1.0, on(ws))),
        ("out", lambda: qm.qm_cache_attend(cache(), batch(), on(x), on(x, gpu), 1.0, on(ws))),
        ("lse", lambda: qm.qm_cache_attend(cache(), batch(), on(x), on(x), 1.0, on(ws), lse=on(lse, gpu))),
        ("workspace", lambda: qm.qm_cache_attend(cache(), batch(), on(x), on(x), 1.0, on(ws, gpu))),
    ]
    if gpu < 0:  # and where everything is on the host
        calls += [("cache", lambda: qm.cache_append(qm.Cache(k, k), qm.Batch(lens, table), x, x)), ("x", lambda: qm.head_norm_rope([x])),
                  ("cache", lambda: qm.cache_attend(qm.Cache(k, k), qm.Batch(lens, table), x))]
    for part, call in calls:
        with pytest.raises(qm.QMError, match=f"QM_EINVAL: {part}: {why}"):
            call()
    for make in (lambda: qm.Cache(on(k), on(k, gpu)), lambda: qm.Batch(on(lens), on(table, gpu)), lambda: qm.Batch(on(lens, gpu), on(table)),
                 lambda: qm.Batch(on(lens), on(table), on(torch.zeros(3, dtype=torch.int32), gpu))):
        with pytest.raises(qm.QMError, match="must be on one device"):
            make()
