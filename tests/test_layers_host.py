"""Refusals of the epilogues, the router and the sum over experts, on the host: every
case fails validation before any CUDA call and names the part."""
import ctypes
import math

import pytest
import torch

import packed_qmatmul_gb300 as qm

A = 1 << 20  # an aligned address nothing reads


@pytest.fixture(scope="module")
def lib():
    from packed_qmatmul_gb300 import build

    build.build()
    return qm.load_library()


def refused(lib, st, part, status=qm.QM_EINVAL):
    msg = lib.qm_last_error().decode()
    assert st == status and msg.startswith(part), (st, msg)


def weight(shape=(16, 64), ndim=2):
    w = qm._CWeight()
    w.format, w.bits, w.group_size, w.scale_dtype, w.ndim = qm.QM_AFFINE, 4, 64, qm.QM_BF16, ndim
    for i, s in enumerate(shape):
        w.shape[i] = s
    w.codes, w.scales, w.biases = 256, 512, 768
    return w


def epilogue(bias=0, residual=0, stride=0, bias_dtype=qm.QM_BF16, act=0, gated=0, alpha=1.0, limit=0.0, up=0.0):
    return qm._EPILOGUE(bias, residual, stride, bias_dtype, act, gated, alpha, limit, up)


def router(bias=0, experts=64, topk=4, score=0, groups=1, topk_groups=1, group_score=0, renormalize=1, scale=1.0):
    return qm._ROUTER(bias, experts, topk, score, groups, topk_groups, group_score, renormalize, scale)


def test_struct_sizes():
    assert [len(epilogue()), len(router())] == [48, 40]


EPILOGUES = [
    ("epilogue", None), ("epilogue", dict(act=-1)), ("epilogue", dict(act=5)), ("epilogue", dict(gated=2)), ("epilogue", dict(act=2, alpha=math.nan)),
    ("epilogue", dict(act=2, alpha=math.inf)), ("epilogue", dict(gated=1, limit=-1.0)), ("epilogue", dict(gated=1, limit=math.nan)),
    ("epilogue", dict(gated=1, up=math.inf)), ("epilogue", dict(limit=1.0)), ("epilogue", dict(up=1.0)), ("bias", dict(bias=A, bias_dtype=qm.QM_I8)),
    ("bias", dict(bias=A + 2)),
]


@pytest.mark.parametrize("part,change", EPILOGUES + [
    ("residual", dict(residual=A + 1, stride=16)), ("residual", dict(residual=A, stride=-16)), ("residual", dict(residual=A, stride=1 << 62)),
    ("residual", dict(residual=8192 + 2, stride=16)), ("residual", dict(residual=8192, stride=32)), ("residual", dict(residual=8192 - 64, stride=16)),
    ("bias", dict(bias=8192 + 16)), ("bias", dict(bias=8192 - 16)),
])
def test_apply_fused_refusals(lib, part, change):
    ep = None if change is None else epilogue(**change)
    refused(lib, lib.qm_apply_fused(ctypes.byref(weight()), 4096, 3, qm.QM_BF16, ep, 8192, None), part)


@pytest.mark.parametrize("part,status,args", [
    ("w", qm.QM_EINVAL, dict(w=weight((15, 64)), ep=epilogue(gated=1))), ("w", qm.QM_ENOTSUP, dict(w=weight((2, 16, 64), 3))),
    ("x", qm.QM_EINVAL, dict(M=-1)), ("x", qm.QM_ENOTSUP, dict(dt=qm.QM_F16)), ("y", qm.QM_EINVAL, dict(y=0)), ("y", qm.QM_EINVAL, dict(y=8192 + 8)),
    ("y", qm.QM_EINVAL, dict(y=4096 + 16)), ("x", qm.QM_EINVAL, dict(x=0)), ("x", qm.QM_EINVAL, dict(x=4096 + 2)), ("w", qm.QM_EINVAL, dict(w=None)),
])
def test_apply_fused_product_refusals(lib, part, status, args):
    a = dict(w=weight(), x=4096, M=3, dt=qm.QM_BF16, ep=epilogue(act=1), y=8192) | args
    w = None if a["w"] is None else ctypes.byref(a["w"])
    refused(lib, lib.qm_apply_fused(w, a["x"], a["M"], a["dt"], a["ep"], a["y"], None), part, status)


def test_apply_fused_takes_nothing(lib):
    assert lib.qm_apply_fused(ctypes.byref(weight()), None, 0, qm.QM_BF16, epilogue(act=1), None, None) == qm.QM_OK
    assert lib.qm_apply_fused(ctypes.byref(weight((0, 64))), 4096, 3, qm.QM_BF16, epilogue(gated=1), None, None) == qm.QM_OK


@pytest.mark.parametrize("part,change", EPILOGUES + [("residual", dict(residual=A, stride=16)), ("bias", dict(bias=8192 + 64))])
def test_apply_experts_fused_refusals(lib, part, change):
    ep = None if change is None else epilogue(**change)
    refused(lib, lib.qm_apply_experts_fused(ctypes.byref(weight((2, 16, 64), 3)), A, qm.QM_I32, 3, 2, 4096, 3, qm.QM_BF16, ep, 8192, A, 1 << 16, None), part)


@pytest.mark.parametrize("part,args", [
    ("w", dict(w=weight())), ("w", dict(w=weight((2, 15, 64), 3), ep=epilogue(gated=1))), ("ids", dict(T=-1)), ("ids", dict(ids=0)), ("ids", dict(it=3)),
    ("x", dict(rows=4)), ("y", dict(y=0)), ("workspace", dict(ws=0)), ("workspace", dict(size=16)),
])
def test_apply_experts_fused_product_refusals(lib, part, args):
    a = dict(w=weight((2, 16, 64), 3), ids=A, it=qm.QM_I32, T=3, topk=2, rows=3, y=8192, ws=A, size=1 << 16, ep=epilogue(act=2)) | args
    refused(lib, lib.qm_apply_experts_fused(ctypes.byref(a["w"]), a["ids"], a["it"], a["T"], a["topk"], 4096, a["rows"], qm.QM_BF16, a["ep"], a["y"],
                                            a["ws"], a["size"], None), part)


@pytest.mark.parametrize("part,change", [
    ("router", None), ("router", dict(experts=0)), ("router", dict(experts=1025)), ("router", dict(topk=0)), ("router", dict(topk=32)),
    ("router", dict(experts=3)), ("router", dict(score=2)), ("router", dict(groups=0)), ("router", dict(groups=3)), ("router", dict(groups=64)),
    ("router", dict(groups=4, topk_groups=5)), ("router", dict(topk_groups=0)), ("router", dict(group_score=2)),
    ("router", dict(experts=32, groups=32, group_score=1)), ("router", dict(renormalize=2)), ("router", dict(scale=math.inf)),
    ("router", dict(scale=math.nan)), ("bias", dict(bias=A + 2)), ("bias", dict(bias=4096 + 32)), ("bias", dict(bias=8192 - 128)),
])
def test_router_refusals(lib, part, change):
    r = None if change is None else router(**change)
    refused(lib, lib.qm_experts_select(r, A, qm.QM_F32, 64, 3, 4096, 8192, None), part)


@pytest.mark.parametrize("part,args", [
    ("logits", dict(dt=qm.QM_I8)), ("logits", dict(T=-1)), ("logits", dict(T=1 << 31)), ("logits", dict(stride=-1)), ("logits", dict(logits=0)),
    ("logits", dict(logits=A + 2)), ("logits", dict(logits=A + 1, dt=qm.QM_BF16)), ("logits", dict(stride=1 << 62)), ("ids", dict(ids=0)),
    ("weights", dict(weights=0)), ("ids", dict(ids=4098)), ("weights", dict(weights=8194)), ("ids", dict(ids=8192 + 44)), ("logits", dict(logits=4096 - 700)),
    ("logits", dict(logits=8192 + 40)),
])
def test_select_refusals(lib, part, args):
    a = dict(logits=A, dt=qm.QM_F32, stride=64, T=3, ids=4096, weights=8192) | args
    refused(lib, lib.qm_experts_select(router(), a["logits"], a["dt"], a["stride"], a["T"], a["ids"], a["weights"], None), part)


def test_select_takes_nothing(lib):
    assert lib.qm_experts_select(router(experts=1020, groups=17, topk_groups=17), None, qm.QM_F32, 1020, 0, None, None, None) == qm.QM_OK


@pytest.mark.parametrize("part,status,args", [
    ("y", qm.QM_ENOTSUP, dict(dt=qm.QM_F32)), ("y", qm.QM_EINVAL, dict(T=-1)), ("y", qm.QM_EINVAL, dict(T=1 << 40, n=1 << 40)), ("y", qm.QM_EINVAL, dict(y=0)),
    ("y", qm.QM_EINVAL, dict(y=A + 8)), ("y", qm.QM_EINVAL, dict(T=1, topk=1 << 32, n=1)), ("weights", qm.QM_EINVAL, dict(weights=0)),
    ("weights", qm.QM_EINVAL, dict(weights=4098)), ("out", qm.QM_EINVAL, dict(out=0)), ("out", qm.QM_EINVAL, dict(out=8192 + 8)),
    ("out", qm.QM_EINVAL, dict(y=8192 - 32)), ("out", qm.QM_EINVAL, dict(weights=8192 + 16)), ("residual", qm.QM_EINVAL, dict(residual=A + 1)),
    ("residual", qm.QM_EINVAL, dict(residual=8192 + 16)), ("residual", qm.QM_EINVAL, dict(residual=8192, stride=8)),
    ("residual", qm.QM_EINVAL, dict(residual=A, stride=-16)),
])
def test_combine_refusals(lib, part, status, args):
    a = dict(y=A, weights=4096, T=3, topk=2, n=16, dt=qm.QM_BF16, residual=0, stride=16, out=8192) | args
    refused(lib, lib.qm_experts_combine(a["y"], a["weights"], a["T"], a["topk"], a["n"], a["dt"], a["residual"], a["stride"], a["out"], None), part, status)


def test_combine_takes_nothing(lib):
    assert lib.qm_experts_combine(None, None, 0, 2, 16, qm.QM_BF16, None, 0, None, None) == qm.QM_OK


# ---------------------------------------------------------------- the binding's own
def qweight(shape):
    k = shape[-1]
    lead = shape[:-1]
    return qm.QWeight("affine", shape, torch.zeros(*lead, k // 2, dtype=torch.uint8), torch.zeros(*lead, k // 64, dtype=torch.bfloat16),
                      torch.zeros(*lead, k // 64, dtype=torch.bfloat16), bits=4, group_size=64)


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("part,call", [
    ("epilogue", lambda: qm.Epilogue(act="swish")), ("bias", lambda: qm.Epilogue(bias=torch.zeros(4, dtype=torch.int32))),
    ("epilogue", lambda: qm.Epilogue(act="silu", alpha=0.0)),
    ("bias", lambda: qm.apply_fused(qweight((16, 64)), bf(3, 64), qm.Epilogue(bias=bf(15)))),
    ("w", lambda: qm.apply_fused(qweight((2, 16, 64)), bf(3, 64), qm.Epilogue())),
    ("x", lambda: qm.apply_fused(qweight((16, 64)), bf(3, 32), qm.Epilogue())),
    ("x", lambda: qm.apply_fused(qweight((16, 64)), bf(64), qm.Epilogue())),
    ("x", lambda: qm.apply_fused(qweight((16, 64)), torch.zeros(3, 64), qm.Epilogue())),
    ("x", lambda: qm.apply_fused(qweight((16, 64)), bf(3, 64), qm.Epilogue())),  # not on a GPU
    ("residual", lambda: qm.apply_fused(qweight((16, 64)), bf(3, 64), qm.Epilogue(), bf(3, 8))),
    ("residual", lambda: qm.apply_fused(qweight((16, 64)), bf(3, 64), qm.Epilogue(gated=True), bf(3, 16))),
    ("residual", lambda: qm.apply_fused(qweight((16, 64)), bf(3, 64), qm.Epilogue(), bf(16, 3).T)),
    ("y", lambda: qm.qm_apply_fused(qweight((16, 64)), bf(3, 64), qm.Epilogue(gated=True), bf(3, 16))),
    ("bias", lambda: qm.apply_experts_fused(qweight((2, 16, 64)), torch.zeros(3, 2, dtype=torch.int32), bf(3, 64), qm.Epilogue(bias=bf(16)))),
    ("ids", lambda: qm.apply_experts_fused(qweight((2, 16, 64)), torch.zeros(6, dtype=torch.int32), bf(3, 64), qm.Epilogue())),
    ("ids", lambda: qm.apply_experts_fused(qweight((2, 16, 64)), torch.zeros(3, 2), bf(3, 64), qm.Epilogue())),
    ("x", lambda: qm.apply_experts_fused(qweight((2, 16, 64)), torch.zeros(3, 2, dtype=torch.int32), bf(4, 64), qm.Epilogue())),
    ("router", lambda: qm.Router(2, score="tanh")), ("router", lambda: qm.Router(2, group_score="mean")), ("bias", lambda: qm.Router(2, bias=bf(8))),
    ("bias", lambda: qm.experts_select(torch.zeros(3, 8), qm.Router(2, bias=torch.zeros(9)))),
    ("logits", lambda: qm.experts_select(torch.zeros(8), qm.Router(2))), ("logits", lambda: qm.experts_select(torch.zeros(3, 8).double(), qm.Router(2))),
    ("logits", lambda: qm.experts_select(torch.zeros(8, 3).T, qm.Router(2))), ("logits", lambda: qm.experts_select(torch.zeros(3, 8), qm.Router(2))),
    ("ids", lambda: qm.qm_experts_select(torch.zeros(3, 8), qm.Router(2), torch.zeros(3, 2), torch.zeros(3, 2))),
    ("weights", lambda: qm.qm_experts_select(torch.zeros(3, 8), qm.Router(2), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 3))),
    ("y", lambda: qm.experts_combine(bf(3, 16), torch.zeros(3, 2))), ("weights", lambda: qm.experts_combine(bf(3, 2, 16), bf(3, 2))),
    ("residual", lambda: qm.experts_combine(bf(3, 2, 16), torch.zeros(3, 2), bf(2, 16))), ("y", lambda: qm.experts_combine(bf(3, 2, 16), torch.zeros(3, 2))),
    ("out", lambda: qm.qm_experts_combine(bf(3, 2, 16), torch.zeros(3, 2), bf(3, 8))),
])
def test_binding_refusals(lib, part, call):
    with pytest.raises(qm.QMError) as e:
        call()
    assert e.value.status == qm.QM_EINVAL and e.value.message.startswith(part), e.value.message
