"""GB300-native weight-only quantized products over packed block formats.

A thin ctypes binding over libqm (include/qm.h). Every function marshals its
arguments and calls the C entry point of the same name; every step of the
work runs in the library's CUDA kernels. PyTorch supplies device memory and
the current stream. There is no CPU fallback: if libqm.so is missing or fails
to load, the first call raises.

Formats (see include/qm.h): MLX affine (uint32 codes + per-group scales and
biases), GGUF Q8_0 (34-byte blocks of 32 values) and MXFP4 (e2m1 codes, two
per byte, plus e8m0 scales per 32 values).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct
import threading
from typing import Optional, Sequence

import torch

__all__ = [
    "QM_AFFINE", "QM_Q8_0", "QM_MXFP4", "QM_MXFP4_BLOCKS", "QM_Q4_K", "QM_Q6_K", "QM_WEIGHT_STATIC", "QM_F32", "QM_BF16", "QM_F16", "QM_I8", "QM_I32", "QM_I64",
    "QM_ROPE_HALF", "QM_ROPE_PAIRS",
    "QMError", "QWeight", "Rope", "Cache", "Batch", "library_path", "load_library",
    "qm_dequant", "qm_quantize_q8_0", "qm_apply", "qm_apply_many", "qm_take", "qm_apply_experts", "qm_apply_experts_workspace",
    "qm_experts_route_workspace",
    "qm_experts_route", "qm_apply_experts_static", "qm_check_wait_timeout", "qm_device_status", "qm_last_error",
    "qm_version", "qm_head_norm_rope", "qm_cache_append", "qm_cache_attend", "qm_cache_attend_workspace",
    "dequant", "quantize_q8_0", "apply", "apply_many", "take", "apply_experts", "route",
    "head_norm_rope", "cache_append", "cache_attend",
]

QM_OK, QM_EINVAL, QM_ECUDA, QM_ETIMEOUT, QM_ENOTSUP = 0, 1, 2, 3, 4
QM_AFFINE, QM_Q8_0, QM_MXFP4, QM_MXFP4_BLOCKS, QM_Q4_K, QM_Q6_K = 0, 1, 2, 3, 4, 5
QM_F32, QM_BF16, QM_F16, QM_I8 = 0, 1, 2, 3
QM_ROPE_HALF, QM_ROPE_PAIRS = 0, 1
QM_I32, QM_I64 = 0, 1
QM_WEIGHT_STATIC = 1
QM_MAX_NDIM = 4
QM_MAX_MANY = 8
QM_MAX_HEAD_SETS = 4

_STATUS = {QM_EINVAL: "QM_EINVAL", QM_ECUDA: "QM_ECUDA", QM_ETIMEOUT: "QM_ETIMEOUT",
           QM_ENOTSUP: "QM_ENOTSUP"}
_FORMATS = {"affine": QM_AFFINE, "q8_0": QM_Q8_0, "mxfp4": QM_MXFP4, "mxfp4_blocks": QM_MXFP4_BLOCKS,
            "q4_k": QM_Q4_K, "q6_k": QM_Q6_K}
_DTYPES = {torch.float32: QM_F32, torch.bfloat16: QM_BF16, torch.float16: QM_F16}
_ITYPES = {torch.int32: QM_I32, torch.int64: QM_I64}
_CACHE_DTYPES = {torch.bfloat16: QM_BF16, torch.float16: QM_F16, torch.int8: QM_I8}

_HERE = os.path.dirname(os.path.abspath(__file__))
_lock = threading.Lock()
_lib = None


class QMError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS.get(status, status)}: {message}")
        self.status = status
        self.message = message


class _CWeight(ctypes.Structure):
    _fields_ = [
        ("format", ctypes.c_int32), ("bits", ctypes.c_int32), ("group_size", ctypes.c_int32),
        ("scale_dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
        ("shape", ctypes.c_int64 * QM_MAX_NDIM),
        ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("biases", ctypes.c_void_p),
        ("flags", ctypes.c_uint32),
    ]


def library_path() -> str:
    return os.environ.get("QM_LIBRARY") or os.path.join(_HERE, "libqm.so")


def load_library():
    """Loads libqm.so (built by packed_qmatmul_gb300/build.py); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"libqm.so not found at {path}: run "
                               "`python -c 'import __graft_entry__ as g; g.build()'` first")
        lib = ctypes.CDLL(path)
        i32, i64, vp, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
        wp = ctypes.POINTER(_CWeight)
        sigs = {
            "qm_dequant": ([wp, i32, vp, vp], i32),
            "qm_quantize_q8_0": ([vp, i32, i64, i64, vp, vp], i32),
            "qm_check_wait_timeout": ([ctypes.c_uint64, vp], i32),
            "qm_apply": ([wp, vp, i64, i32, vp, vp], i32),
            "qm_apply_many": ([ctypes.POINTER(wp), i32, vp, i64, i32, ctypes.POINTER(vp), vp], i32),
            "qm_take": ([wp, i32, vp, i32, i64, vp, vp, vp, i32, vp, vp], i32),
            "qm_apply_experts_workspace": ([wp, i64, i64], sz),
            "qm_experts_route_workspace": ([i64, i64], sz),
            "qm_apply_experts": ([wp, vp, i32, i64, i64, vp, i64, i32, vp, vp, sz, vp], i32),
            "qm_experts_route": ([vp, i32, i64, i64, vp, vp, vp, vp, sz, vp], i32),
            "qm_apply_experts_static": ([wp, vp, i32, i64, i64, vp, i64, i32, vp, vp], i32),
            "qm_head_norm_rope": ([vp, vp, vp, i32, i64, i32, ctypes.c_float, vp, vp, i32, vp], i32),
            "qm_cache_append": ([vp, vp, vp, vp, vp, ctypes.c_float, vp, vp], i32),
            "qm_cache_attend_workspace": ([vp, vp, i32], sz),
            "qm_cache_attend": ([vp, vp, vp, vp, vp, ctypes.c_float, i64, vp, sz, vp], i32),
            "qm_device_status": ([vp], i32),
            "qm_last_error": ([], ctypes.c_char_p),
            "qm_version": ([], i32),
        }
        for name, (args, res) in sigs.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
        return lib


def _check(status: int):
    if status != QM_OK:
        msg = load_library().qm_last_error().decode()
        raise QMError(status, msg)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("libqm takes contiguous tensors")
    return t.data_ptr()


# The current stream's handle without building a Stream object (0.3 against 2.9 us of a call's host time).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> Optional[int]:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _on(stream):
    """Where a call's own tensors are allocated: on the stream that uses them (the caching allocator hands
    out again what is freed on a stream as soon as that stream's earlier work is enqueued)."""
    if stream is None:
        return _HERE_NOW
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


_HERE_NOW = contextlib.nullcontext()


# ---------------------------------------------------------------- weights
class QWeight:
    """A packed weight: format, logical shape [..., n, k] and device parts.

    Parts are device tensors whose bytes are the format's (any integer dtype of
    the right byte size; uint32 codes may be held as int32). The descriptor
    passed to the library is built once and rebuilt when a field is assigned;
    parts are read through their tensors' addresses at that time.
    """

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name != "_cref":
            object.__setattr__(self, "_cref", None)

    def __init__(self, fmt, shape: Sequence[int], codes: torch.Tensor,
                 scales: Optional[torch.Tensor] = None, biases: Optional[torch.Tensor] = None,
                 bits: int = 0, group_size: int = 0, scale_dtype: int = QM_BF16, flags: int = 0):
        self.format = _FORMATS[fmt] if isinstance(fmt, str) else int(fmt)
        self.shape = tuple(int(s) for s in shape)
        self.codes, self.scales, self.biases = codes, scales, biases
        self.bits = int(bits)
        self.group_size = int(group_size)
        self.scale_dtype = int(scale_dtype)
        self.flags = int(flags)

    @classmethod
    def from_arrays(cls, d: dict, device="cuda", flags: int = 0) -> "QWeight":
        """From a dict of NumPy parts as packed_qmatmul_gb300.synth returns."""
        import numpy as np

        def dev(a):
            if a is None:
                return None
            a = np.ascontiguousarray(a)
            view = {np.dtype(np.uint32): np.int32, np.dtype(np.uint16): np.int16}.get(a.dtype)
            t = torch.from_numpy(a.view(view) if view is not None else a)
            return t.to(device)

        sdt = QM_F16 if d.get("scale_dtype") == "f16" else QM_BF16
        return cls(d["format"], d["shape"], dev(d["codes"]), dev(d.get("scales")),
                   dev(d.get("biases")), bits=d.get("bits", 0), group_size=d.get("group_size", 0),
                   scale_dtype=sdt, flags=flags)

    def _ref(self):
        """ctypes reference to the descriptor (cached)."""
        ref = self._cref
        if ref is None:
            ref = ctypes.byref(self._c())
            object.__setattr__(self, "_cref", ref)
        return ref

    def _pointer(self):
        """ctypes pointer to the same cached descriptor (for arrays of weights)."""
        ref = self._ref()
        cached = self.__dict__.get("_cptr")
        if cached is None or cached[0] is not ref:  # the descriptor was rebuilt
            cached = (ref, ctypes.pointer(ref._obj))
            object.__setattr__(self, "_cptr", cached)
        return cached[1]

    def _c(self) -> _CWeight:
        w = _CWeight()
        w.format, w.bits, w.group_size, w.scale_dtype = (self.format, self.bits, self.group_size,
                                                          self.scale_dtype)
        w.ndim = len(self.shape)
        for i, s in enumerate(self.shape[:QM_MAX_NDIM]):
            w.shape[i] = s
        w.codes, w.scales, w.biases = _ptr(self.codes), _ptr(self.scales), _ptr(self.biases)
        w.flags = self.flags
        return w

    def part_shapes(self, lead: Sequence[int]):
        """Byte shapes of (codes, scales, biases) for leading dims `lead` + [n]."""
        k = self.shape[-1]
        if self.format == QM_AFFINE:
            cb, sb = k * self.bits // 8, k // self.group_size * 2
            return (tuple(lead) + (cb,), tuple(lead) + (sb,), tuple(lead) + (sb,))
        if self.format == QM_Q8_0:
            return (tuple(lead) + (k // 32 * 34,), None, None)
        if self.format == QM_MXFP4_BLOCKS:
            return (tuple(lead) + (k // 32 * 17,), None, None)
        if self.format == QM_Q4_K:
            return (tuple(lead) + (k // 256 * 144,), None, None)
        if self.format == QM_Q6_K:
            return (tuple(lead) + (k // 256 * 210,), None, None)
        return (tuple(lead) + (k // 2,), tuple(lead) + (k // 32,), None)


# ---------------------------------------------------------------- heads and the paged cache
# C descriptors as packed bytes, in include/qm.h's order; a bytes object passes
# as a pointer to them.
_HEADS = struct.Struct("Pqqii").pack
_ROPE = struct.Struct("Pqii").pack
_CACHE = struct.Struct("4P7q4i").pack
_BATCH = struct.Struct("3P3q2i").pack
_POINTERS = [struct.Struct(f"{i}P").pack for i in range(QM_MAX_HEAD_SETS + 1)]


def _refuse(message: str):
    raise QMError(QM_EINVAL, message)


def _heads(x: torch.Tensor, tokens: int, heads: int, dim: int, name: str) -> bytes:
    """The descriptor of x [tokens, heads, dim] (its last axis contiguous, the others strided as they are)."""
    if x.shape != (tokens, heads, dim):
        _refuse(f"{name}: shape {tuple(x.shape)}, expected {(tokens, heads, dim)}")
    ts, hs, es = x.stride()
    if es != 1 and dim > 1:
        _refuse(f"{name}: the elements of a head must be contiguous")
    return _HEADS(x.data_ptr(), ts, hs, heads, _DTYPES.get(x.dtype, -1))


def _heads_and_like(x: torch.Tensor, tokens: int, dim: int, name: str):
    """x's descriptor, a new contiguous tensor of its shape and type, and that one's descriptor."""
    shape = x.shape
    if len(shape) != 3 or shape[0] != tokens or shape[2] != dim:
        _refuse(f"{name}: shape {tuple(shape)}, expected {(tokens, 'heads', dim)}")
    heads = shape[1]
    ts, hs, es = x.stride()
    if es != 1 and dim > 1:
        _refuse(f"{name}: the elements of a head must be contiguous")
    dtype = x.dtype
    code = _DTYPES.get(dtype, -1)
    row = heads * dim
    y = torch.empty_like(x) if hs == dim and ts == row else torch.empty(shape, dtype=dtype, device=x.device)
    return _HEADS(x.data_ptr(), ts, hs, heads, code), y, _HEADS(y.data_ptr(), row, dim, heads, code)


def _one_gpu(gpus: Sequence[Optional[int]], names: Sequence[str]):
    """Refuses a call whose tensors are not on one GPU, where a kernel would read a host tensor's address as its
    own. gpus: each part's get_device(), None for a part that the call goes without."""
    gpu = gpus[0]
    if gpu < 0 or gpus.count(gpu) + gpus.count(None) != len(gpus):
        for g, name in zip(gpus, names):
            if g is not None and (g < 0 or g != gpu):
                _refuse(f"{name}: {'not on a GPU' if g < 0 else 'on another GPU than ' + names[0]}")


def _gpu(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.get_device()


def _i32(t: torch.Tensor, name: str) -> int:
    if t.dtype != torch.int32:
        _refuse(f"{name}: must be int32")
    return _ptr(t)


class Rope:
    """A rotation of a head's first elements by position (qm_rope): `table` float32
    [rows, dim], row p the dim/2 cosines then the dim/2 sines of position p; style
    "half" pairs elements (i, i + dim/2), "pairs" (2i, 2i + 1)."""

    def __init__(self, table: torch.Tensor, style: str = "half"):
        if table.dtype != torch.float32 or table.dim() != 2:
            _refuse("rope: table must be float32 [rows, dim]")
        if style not in ("half", "pairs"):
            _refuse('rope: style must be "half" or "pairs"')
        self.table, self.style = table, style
        self.dim = table.shape[1]
        self.gpu = table.get_device()
        self._c = _ROPE(_ptr(table), table.shape[0], self.dim, QM_ROPE_HALF if style == "half" else QM_ROPE_PAIRS)


class Cache:
    """A paged key/value cache (qm_cache): k and v [pages, heads, page_size, dim],
    bfloat16 or float16, or int8 codes with float32 k_scales and v_scales [pages,
    heads, page_size]. Any strides whose last axis is contiguous do (a cache laid
    out [pages, page_size, heads, dim] is passed permuted), the same for k and v.
    The descriptor is built here, from the tensors' addresses at that time."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scales: Optional[torch.Tensor] = None,
                 v_scales: Optional[torch.Tensor] = None):
        if k.dim() != 4 or v.shape != k.shape or v.dtype != k.dtype:
            _refuse("cache: k and v must be [pages, heads, page_size, dim] of one shape and dtype")
        if k.dtype not in _CACHE_DTYPES:
            _refuse("cache: dtype must be bfloat16, float16 or int8")
        if k.stride() != v.stride() or (k.stride(3) != 1 and k.shape[3] > 1):
            _refuse("cache: k and v must have the same strides and contiguous heads")
        scales = (k_scales, v_scales)
        if any((s is None) != (k.dtype != torch.int8) for s in scales):
            _refuse("k_scales: an int8 cache has k_scales and v_scales, another has neither")
        sst = (0, 0, 0)
        if k.dtype == torch.int8:
            if any(s.dtype != torch.float32 or s.shape != k.shape[:3] for s in scales) or k_scales.stride() != v_scales.stride():
                _refuse("k_scales: scales must be float32 [pages, heads, page_size] of the same strides")
            sst = k_scales.stride()
        self.gpu = k.get_device()
        if any(s is not None and s.get_device() != self.gpu for s in (v, *scales)):
            _refuse("cache: its tensors must be on one device")
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.pages, self.heads, self.page_size, self.dim = k.shape
        self._need = {}
        self._c = _CACHE(k.data_ptr(), v.data_ptr(), *(0 if s is None else s.data_ptr() for s in scales), *k.stride()[:3],
                         *sst, self.pages, _CACHE_DTYPES[k.dtype], self.heads, self.dim, self.page_size)


class Batch:
    """The new tokens of a call (qm_batch): lens int32 [seqs] (tokens of each sequence
    with the new ones; 0: an empty slot), page_table int32 [seqs, width], q_offsets
    int32 [seqs + 1] where each sequence's rows begin (None: tokens / seqs rows
    each), `tokens` the rows in all (None: seqs), max_new the most new tokens of a sequence
    if known. The tensors may be updated in place between calls."""

    def __init__(self, lens: torch.Tensor, page_table: torch.Tensor, q_offsets: Optional[torch.Tensor] = None,
                 tokens: Optional[int] = None, max_new: int = 0):
        seqs = lens.shape[0]
        if lens.dim() != 1 or page_table.dim() != 2 or page_table.shape[0] != seqs:
            _refuse("batch: lens must be [seqs] and page_table [seqs, width]")
        if q_offsets is not None and q_offsets.shape != (seqs + 1,):
            _refuse("q_offsets: must be [seqs + 1]")
        if page_table.dtype != torch.int32 or (page_table.stride(1) != 1 and page_table.shape[1] > 1):
            _refuse("page_table: must be int32 with contiguous rows")
        self.gpu = lens.get_device()
        if page_table.get_device() != self.gpu or (q_offsets is not None and q_offsets.get_device() != self.gpu):
            _refuse("batch: its tensors must be on one device")
        self.lens, self.page_table, self.q_offsets = lens, page_table, q_offsets
        self.seqs, self.tokens, self.max_new = seqs, seqs if tokens is None else int(tokens), int(max_new)
        self._c = _BATCH(_i32(lens, "lens"), page_table.data_ptr(), 0 if q_offsets is None else _i32(q_offsets, "q_offsets"),
                         self.tokens, page_table.shape[1], page_table.stride(0), seqs, self.max_new)


# ---------------------------------------------------------------- C entry points
def qm_version() -> int:
    return load_library().qm_version()


def qm_last_error() -> str:
    return load_library().qm_last_error().decode()


def qm_dequant(w: QWeight, out: torch.Tensor, stream=None) -> None:
    _check(load_library().qm_dequant(w._ref(), _DTYPES[out.dtype], _ptr(out),
                                     _stream(stream)))


def qm_quantize_q8_0(x: torch.Tensor, blocks: torch.Tensor, stream=None) -> None:
    k = x.shape[-1]
    rows = x.numel() // k if k else 0
    _check(load_library().qm_quantize_q8_0(_ptr(x), _DTYPES[x.dtype], rows, k, _ptr(blocks),
                                           _stream(stream)))


def qm_apply(w: QWeight, x: torch.Tensor, y: torch.Tensor, stream=None) -> None:
    M = x.shape[0] if x.dim() == 2 else 1
    _check(load_library().qm_apply(w._ref(), _ptr(x), M, _DTYPES[x.dtype], _ptr(y),
                                   _stream(stream)))


_WARR = [ctypes.POINTER(_CWeight) * max(i, 1) for i in range(QM_MAX_MANY + 1)]
_PARR = [ctypes.c_void_p * max(i, 1) for i in range(QM_MAX_MANY + 1)]


_MANY = {}


def _weight_array(ws):
    """The C array of descriptor pointers for these weights, kept per tuple of
    weights and rebuilt when any of their descriptors was (a cached entry holds
    its descriptors, so a weight reusing an id cannot match a stale one)."""
    key = tuple(map(id, ws))
    hit = _MANY.get(key)
    if hit is not None and tuple([w._cref for w in ws]) == hit[0]:  # descriptors compare by identity
        return hit[1]
    refs = tuple(w._ref() for w in ws)
    arr = _WARR[len(ws)](*[w._pointer() for w in ws])
    if len(_MANY) >= 1024:
        _MANY.clear()
    _MANY[key] = (refs, arr)
    return arr


def qm_apply_many(ws: Sequence[QWeight], x: torch.Tensor, ys: Sequence[torch.Tensor], stream=None) -> None:
    """ys[i] = x times ws[i]^T for weights that read the same x (one launch at M = 1)."""
    M = x.shape[0] if x.dim() == 2 else 1
    n = len(ws)
    if n > QM_MAX_MANY or len(ys) != n:  # the C call refuses these; keep the arrays in range
        raise QMError(QM_EINVAL, f"count: {n} weights and {len(ys)} outputs (1 .. {QM_MAX_MANY} each)")
    warr = _weight_array(ws)
    yarr = _PARR[n](*[_ptr(y) for y in ys])
    _check(load_library().qm_apply_many(warr, n, _ptr(x), M, _DTYPES[x.dtype], yarr, _stream(stream)))


def qm_take(w: QWeight, axis: int, ids: torch.Tensor, out_codes=None, out_scales=None,
            out_biases=None, out_dense: Optional[torch.Tensor] = None, stream=None) -> None:
    id_type = QM_I64 if ids.dtype == torch.int64 else QM_I32
    out_dtype = _DTYPES[out_dense.dtype] if out_dense is not None else QM_F32
    _check(load_library().qm_take(w._ref(), axis, _ptr(ids), id_type, ids.numel(),
                                  _ptr(out_codes), _ptr(out_scales), _ptr(out_biases), out_dtype,
                                  _ptr(out_dense), _stream(stream)))


def qm_apply_experts_workspace(w: QWeight, T: int, topk: int) -> int:
    return load_library().qm_apply_experts_workspace(w._ref(), T, topk)


def qm_experts_route_workspace(P: int, E: int) -> int:
    return load_library().qm_experts_route_workspace(P, E)


def qm_apply_experts(w: QWeight, ids: torch.Tensor, x: torch.Tensor, y: torch.Tensor,
                     workspace: torch.Tensor, stream=None) -> None:
    T, topk = ids.shape
    id_type = QM_I64 if ids.dtype == torch.int64 else QM_I32
    _check(load_library().qm_apply_experts(
        w._ref(), _ptr(ids), id_type, T, topk, _ptr(x), x.shape[0], _DTYPES[x.dtype],
        _ptr(y), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def qm_apply_experts_static(w: QWeight, ids: torch.Tensor, x: torch.Tensor, y: torch.Tensor,
                            stream=None) -> None:
    """qm_apply_experts with the library's own 1 MiB routing scratch (no workspace)."""
    T, topk = ids.shape
    id_type = QM_I64 if ids.dtype == torch.int64 else QM_I32
    _check(load_library().qm_apply_experts_static(
        w._ref(), _ptr(ids), id_type, T, topk, _ptr(x), x.shape[0], _DTYPES[x.dtype],
        _ptr(y), _stream(stream)))


def qm_experts_route(ids: torch.Tensor, E: int, counts: torch.Tensor, offsets: torch.Tensor,
                     perm: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    id_type = QM_I64 if ids.dtype == torch.int64 else QM_I32
    _check(load_library().qm_experts_route(
        _ptr(ids), id_type, ids.numel(), E, _ptr(counts), _ptr(offsets), _ptr(perm),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def _norm_rope(xs, outs, positions, rope, weights, eps, stream) -> list:
    """The call; outs None: new tensors. Returns the outputs."""
    n = len(xs)
    if not 1 <= n <= QM_MAX_HEAD_SETS or (outs is not None and len(outs) != n) or (weights is not None and len(weights) != n):
        _refuse(f"count: 1 .. {QM_MAX_HEAD_SETS} row sets, as many outputs and weights")
    if xs[0].dim() != 3:
        _refuse("x: must be [tokens, heads, dim]")
    T, _, D = xs[0].shape
    xd, od, made = [], [], []
    if outs is None:
        for x in xs:
            c, y, o = _heads_and_like(x, T, D, "x")
            xd.append(c)
            od.append(o)
            made.append(y)
    else:
        for x, y in zip(xs, outs):
            H = x.shape[1]
            xd.append(_heads(x, T, H, D, "x"))
            od.append(_heads(y, T, H, D, "out"))
    warr = None
    if weights is not None:
        shape, dtype = (D,), xs[0].dtype
        for w in weights:
            if w is not None and (w.shape != shape or w.dtype != dtype):
                _refuse("weights: must be [dim] of x's dtype")
        warr = _POINTERS[n](*[0 if w is None else _ptr(w) for w in weights])
    pos, ptype = None, QM_I32
    if positions is not None:
        ptype = _ITYPES.get(positions.dtype)
        if ptype is None or positions.shape != (T,):
            _refuse("positions: must be int32 or int64 [tokens]")
        pos = _ptr(positions)
    gpus = [x.get_device() for x in xs]
    if outs is not None:
        gpus += [y.get_device() for y in outs]
    if weights is not None:
        gpus += [None if w is None else w.get_device() for w in weights]
    if positions is not None:
        gpus.append(positions.get_device())
    if rope is not None:
        gpus.append(rope.gpu)
    if gpus[0] < 0 or gpus.count(gpus[0]) != len(gpus):
        _one_gpu(gpus, ["x"] * n + ["out"] * (n if outs else 0) + ["weights"] * (n if weights else 0) + ["positions"] * (positions is not None) + ["rope"])
    _check(load_library().qm_head_norm_rope(b"".join(xd), b"".join(od), warr, n, T, D, eps, None if rope is None else rope._c,
                                            pos, ptype, _stream(stream)))
    return made


def qm_head_norm_rope(xs: Sequence[torch.Tensor], outs: Sequence[torch.Tensor], positions: Optional[torch.Tensor] = None,
                      rope: Optional[Rope] = None, weights: Optional[Sequence[Optional[torch.Tensor]]] = None,
                      eps: float = 1e-6, stream=None) -> None:
    """outs[i] [tokens, heads_i, dim] = the heads of xs[i] normed by weights[i] and rotated by `positions`."""
    _norm_rope(xs, outs, positions, rope, weights, eps, stream)


def qm_cache_append(cache: Cache, batch: Batch, k: torch.Tensor, v: torch.Tensor, rope: Optional[Rope] = None,
                    k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, stream=None) -> None:
    if k_weight is not None and (k_weight.shape != (cache.dim,) or k_weight.dtype != k.dtype):
        _refuse("k_weight: must be [dim] of k's dtype")
    kd, vd = _heads(k, batch.tokens, cache.heads, cache.dim, "k"), _heads(v, batch.tokens, cache.heads, cache.dim, "v")
    _one_gpu((cache.gpu, batch.gpu, k.get_device(), v.get_device(), _gpu(k_weight), None if rope is None else rope.gpu),
             ("cache", "batch", "k", "v", "k_weight", "rope"))
    _check(load_library().qm_cache_append(cache._c, batch._c, kd, vd, _ptr(k_weight), eps, None if rope is None else rope._c, _stream(stream)))


def qm_cache_attend_workspace(cache: Cache, batch: Batch, heads: int) -> int:
    key = (batch.seqs, batch.tokens, batch.max_new, heads)  # the shapes that it depends on
    need = cache._need.get(key)
    if need is None:
        if len(cache._need) >= 1024:
            cache._need.clear()
        need = cache._need[key] = load_library().qm_cache_attend_workspace(cache._c, batch._c, heads)
    return need


def qm_cache_attend(cache: Cache, batch: Batch, q: torch.Tensor, out: torch.Tensor, scale: float,
                    workspace: Optional[torch.Tensor], window: int = 0, lse: Optional[torch.Tensor] = None,
                    stream=None) -> None:
    if q.dim() != 3:
        _refuse("q: must be [tokens, heads, dim]")
    T, H = batch.tokens, q.shape[1]
    if lse is not None and (lse.shape != (T, H) or lse.dtype != torch.float32):
        _refuse("lse: must be float32 [tokens, heads]")
    qd, od = _heads(q, T, H, cache.dim, "q"), _heads(out, T, H, cache.dim, "out")
    _one_gpu((cache.gpu, batch.gpu, q.get_device(), out.get_device(), _gpu(lse), _gpu(workspace)),
             ("cache", "batch", "q", "out", "lse", "workspace"))
    _check(load_library().qm_cache_attend(
        cache._c, batch._c, qd, od, _ptr(lse), scale, window, _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream)))


def qm_check_wait_timeout(limit_ns: int, stream=None) -> None:
    _check(load_library().qm_check_wait_timeout(limit_ns, _stream(stream)))


def qm_device_status(stream=None) -> None:
    _check(load_library().qm_device_status(_stream(stream)))


# ---------------------------------------------------------------- conveniences
def dequant(w: QWeight, dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    out = torch.empty(w.shape, dtype=dtype, device=w.codes.device)
    qm_dequant(w, out, stream)
    return out


def quantize_q8_0(x: torch.Tensor, stream=None) -> QWeight:
    """The float weight x [..., n, k] (float32, bfloat16 or float16) stored as GGUF Q8_0."""
    k = x.shape[-1]
    blocks = torch.empty(tuple(x.shape[:-1]) + (k // 32 * 34,), dtype=torch.uint8, device=x.device)
    qm_quantize_q8_0(x, blocks, stream)
    return QWeight("q8_0", tuple(x.shape), blocks)


def apply(w: QWeight, x: torch.Tensor, stream=None) -> torch.Tensor:
    y = torch.empty((x.shape[0], w.shape[-2]), dtype=x.dtype, device=x.device)
    qm_apply(w, x, y, stream)
    return y


def apply_many(ws: Sequence[QWeight], x: torch.Tensor, stream=None) -> list:
    ys = [torch.empty((x.shape[0], w.shape[-2]), dtype=x.dtype, device=x.device) for w in ws]
    qm_apply_many(ws, x, ys, stream)
    return ys


def take(w: QWeight, axis: int, ids: torch.Tensor, dense_dtype=None, packed=True, stream=None):
    """Returns (packed QWeight or None, dense tensor or None)."""
    ndim = len(w.shape)
    ax = axis + ndim if axis < 0 else axis
    n = ids.numel()
    out_shape = w.shape[:ax] + (n,) + w.shape[ax + 1:]
    dev = w.codes.device
    outs = [None, None, None]
    tw = None
    if packed:
        shapes = w.part_shapes(out_shape[:-1])
        outs = [None if s is None else torch.empty(s, dtype=torch.uint8, device=dev) for s in shapes]
        tw = QWeight(w.format, out_shape, outs[0], outs[1], outs[2], bits=w.bits,
                     group_size=w.group_size, scale_dtype=w.scale_dtype)
    dense = None if dense_dtype is None else torch.empty(out_shape, dtype=dense_dtype, device=dev)
    qm_take(w, axis, ids, outs[0], outs[1], outs[2], dense, stream)
    return tw, dense


def apply_experts(w: QWeight, ids: torch.Tensor, x: torch.Tensor, stream=None) -> torch.Tensor:
    T, topk = ids.shape
    y = torch.empty((T, topk, w.shape[-2]), dtype=x.dtype, device=x.device)
    ws = torch.empty(max(qm_apply_experts_workspace(w, T, topk), 256), dtype=torch.uint8,
                     device=x.device)
    qm_apply_experts(w, ids, x, y, ws, stream)
    return y


def route(ids: torch.Tensor, E: int, stream=None):
    P = ids.numel()
    dev = ids.device
    counts = torch.empty(max(E, 1), dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    perm = torch.empty(max(P, 1), dtype=torch.int32, device=dev)
    ws = torch.empty(max(qm_experts_route_workspace(P, E), 256), dtype=torch.uint8, device=dev)
    qm_experts_route(ids, E, counts, offsets, perm, ws, stream)
    return counts[:E], offsets, perm[:P]


def head_norm_rope(xs: Sequence[torch.Tensor], positions: Optional[torch.Tensor] = None, rope: Optional[Rope] = None,
                   weights: Optional[Sequence[Optional[torch.Tensor]]] = None, eps: float = 1e-6, stream=None) -> list:
    """Every head of xs[i] [tokens, heads_i, dim] (queries, keys: any strided rows) normed by weights[i] [dim] and
    rotated by its token's position. qm_head_norm_rope takes outs and allocates nothing."""
    with _on(stream):
        return _norm_rope(xs, None, positions, rope, weights, eps, stream)


def cache_append(cache: Cache, batch: Batch, k: torch.Tensor, v: torch.Tensor, rope: Optional[Rope] = None,
                 k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, stream=None) -> None:
    """Stores the new tokens' keys [tokens, heads, dim] (normed and rotated on the way) and values in the cache."""
    qm_cache_append(cache, batch, k, v, rope, k_weight, eps, stream)


def cache_attend(cache: Cache, batch: Batch, q: torch.Tensor, scale: Optional[float] = None, window: int = 0,
                 lse: bool = False, workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of the new tokens' queries [tokens, heads, dim] over their sequences in the cache; with lse, (out,
    the scores' log-sum-exp [tokens, heads]). Rows of no sequence are not written: what is returned there is
    uninitialised. qm_cache_attend takes out, lse and workspace and allocates nothing."""
    with _on(stream):
        qd, out, od = _heads_and_like(q, batch.tokens, cache.dim, "q")
        _one_gpu((cache.gpu, batch.gpu, q.get_device(), _gpu(workspace)), ("cache", "batch", "q", "workspace"))
        heads = q.shape[1]
        total = torch.empty((batch.tokens, heads), dtype=torch.float32, device=q.device) if lse else None
        if workspace is None:
            need = qm_cache_attend_workspace(cache, batch, heads)
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
        _check(load_library().qm_cache_attend(
            cache._c, batch._c, qd, od, _ptr(total), cache.dim ** -0.5 if scale is None else scale, window, _ptr(workspace),
            0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream)))
        return (out, total) if lse else out
