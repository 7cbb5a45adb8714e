"""Table-batched embedding (TBE) on GB300: Python binding of ``libtbe_gb300.so``.

The functions here carry the names of the C ABI in ``include/tbe.h`` and only
marshal arguments: torch tensors become device pointers, the current torch
stream becomes the ``stream`` argument, and a nonzero status raises
:class:`TBEError`.  Every step of the operator runs in the library's CUDA
kernels.  If the library has not been built, importing works but the first
call raises; there is no other implementation to fall back on.
"""

from __future__ import annotations

import ctypes
import math
import os
import re
from typing import List, Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtbe_gb300.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "tbe.h")

TBE_OK = 0
TBE_ERR_INVALID_ARG = -1
TBE_ERR_UNSUPPORTED = -2
TBE_ERR_WORKSPACE_TOO_SMALL = -3
TBE_ERR_CUDA = -4
TBE_ERR_INDEX_OOB = -5
TBE_ERR_BAD_OFFSETS = -6
TBE_ERR_TIMEOUT = -7
TBE_ERR_NO_MEMORY = -8

TBE_F32, TBE_F16, TBE_BF16 = 0, 1, 2
TBE_I32, TBE_I64 = 0, 1
TBE_POOL_SUM, TBE_POOL_MEAN = 0, 1
TBE_OPT_SGD, TBE_OPT_ROWWISE_ADAGRAD = 1, 2
TBE_FLAG_NO_HISTOGRAM = 0x1
TBE_FLAG_FORCE_HISTOGRAM = 0x2
TBE_FLAG_SORTED_BACKWARD = 0x4
TBE_FLAG_LENGTH_ORDER = 0x8

PATH_NAMES = {0: "gather", 1: "gather_elementwise", 2: "histogram"}

_DTYPES = {torch.float32: TBE_F32, torch.float16: TBE_F16, torch.bfloat16: TBE_BF16}
_POOL = {"sum": TBE_POOL_SUM, "mean": TBE_POOL_MEAN}


class TBEError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {tbe_strerror(code)} ({code})")


class _Table(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("data", ctypes.c_void_p)]


class _Optimizer(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("lr", ctypes.c_float), ("eps", ctypes.c_float),
                ("state", ctypes.c_void_p)]


class WorkspaceLayout(ctypes.Structure):
    _fields_ = [("sorted_keys", ctypes.c_uint64), ("sorted_vals", ctypes.c_uint64),
                ("uniq", ctypes.c_uint64), ("runstart", ctypes.c_uint64),
                ("num_unique", ctypes.c_uint64), ("total_bytes", ctypes.c_uint64)]


class _AttentionConfig(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("window", ctypes.c_int32), ("sinks", ctypes.c_int32),
                ("scale", ctypes.c_float), ("num_buckets", ctypes.c_int32),
                ("bucket_starts", ctypes.POINTER(ctypes.c_int32))]


class _Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class _Pages(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class _LayerNormConfig(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("dim", ctypes.c_int32), ("eps", ctypes.c_float),
                ("has_weight", ctypes.c_int32), ("has_bias", ctypes.c_int32)]


class _SoftmaxLossConfig(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("dim", ctypes.c_int32), ("scale", ctypes.c_float)]


_lib = None


def library_path() -> str:
    return LIB_PATH


def load_library():
    """Load ``libtbe_gb300.so``; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(LIB_PATH)
    P, i32, i64, u32, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_float
    R, G = ctypes.POINTER(_Rows), ctypes.POINTER(_Pages)
    sig = {
        "tbe_create": ([ctypes.POINTER(_Table), i32, i32, u32, ctypes.POINTER(P)], ctypes.c_int),
        "tbe_destroy": ([P], None),
        "tbe_forward": ([P, P, P, i32, i64, i32, P, P, P], ctypes.c_int),
        "tbe_backward_workspace_bytes": ([P, i64, i32], ctypes.c_size_t),
        "tbe_backward_workspace_layout": ([P, i64, i32, ctypes.POINTER(WorkspaceLayout)], ctypes.c_int),
        "tbe_backward_prepare": ([P, P, P, i32, i64, i32, P, P, ctypes.c_size_t, P], ctypes.c_int),
        "tbe_forward_prepare": ([P, P, P, i32, i64, i32, P, P, P, ctypes.c_size_t, P], ctypes.c_int),
        "tbe_backward_apply": ([P, i64, i32, P, ctypes.POINTER(_Optimizer), P, ctypes.c_size_t, P],
                               ctypes.c_int),
        "tbe_backward_sgd": ([P, P, P, i32, i64, i32, P, P, f32, P, ctypes.c_size_t, P], ctypes.c_int),
        "tbe_backward_rowwise_adagrad": ([P, P, P, i32, i64, i32, P, P, P, f32, f32, P,
                                          ctypes.c_size_t, P], ctypes.c_int),
        "tbe_backward_sgd_noalloc": ([P, P, P, i32, i64, i32, P, P, f32, P], ctypes.c_int),
        "tbe_per_sample_weight_grad": ([P, P, P, i32, i64, i32, P, P, P], ctypes.c_int),
        "tbe_attention_create": ([ctypes.POINTER(_AttentionConfig), ctypes.POINTER(P)], ctypes.c_int),
        "tbe_attention_destroy": ([P], None),
        "tbe_attention_workspace_bytes": ([P, i64, i32, i32], ctypes.c_size_t),
        "tbe_attention_forward": ([P, R, R, R, P, P, i32, i64, i32, P, P, P, ctypes.c_size_t, P], ctypes.c_int),
        "tbe_attention_backward": ([P, R, R, R, P, P, i32, i64, i32, P, P, R, P, P, P, P, P, ctypes.c_size_t, P],
                                   ctypes.c_int),
        "tbe_attention_append": ([P, R, R, P, i32, i64, i32, P, G, G, i32, i32, P, i32, P], ctypes.c_int),
        "tbe_attention_decode_workspace_bytes": ([P, i32, i64], ctypes.c_size_t),
        "tbe_attention_decode": ([P, R, G, G, i32, i32, P, i32, P, i32, i64, P, P, P, ctypes.c_size_t, P],
                                 ctypes.c_int),
        "tbe_attention_get_error": ([P, P], ctypes.c_int),
        "tbe_layer_norm_create": ([ctypes.POINTER(_LayerNormConfig), ctypes.POINTER(P)], ctypes.c_int),
        "tbe_layer_norm_destroy": ([P], None),
        "tbe_layer_norm_forward": ([P, P, i64, P, i64, P, P, i64, P, P, P, P], ctypes.c_int),
        "tbe_layer_norm_workspace_bytes": ([P, i64], ctypes.c_size_t),
        "tbe_layer_norm_backward": ([P, P, i64, P, P, i64, P, i64, P, i64, P, P, P, P, ctypes.c_size_t, P],
                                    ctypes.c_int),
        "tbe_softmax_loss_create": ([ctypes.POINTER(_SoftmaxLossConfig), ctypes.POINTER(P)], ctypes.c_int),
        "tbe_softmax_loss_destroy": ([P], None),
        "tbe_softmax_loss_workspace_bytes": ([P, i64, i64, i32], ctypes.c_size_t),
        "tbe_softmax_loss_forward": ([P, P, i64, P, i64, P, i32, i64, i64, P, P, P, ctypes.c_size_t, P],
                                     ctypes.c_int),
        "tbe_softmax_loss_backward": ([P, P, i64, P, i64, P, i32, i64, i64, P, P, P, P, P, ctypes.c_size_t, P],
                                      ctypes.c_int),
        "tbe_softmax_loss_get_error": ([P, P], ctypes.c_int),
        "tbe_get_error": ([P, P], ctypes.c_int),
        "tbe_strerror": ([ctypes.c_int], ctypes.c_char_p),
        "tbe_last_cuda_error": ([], ctypes.c_int),
        "tbe_table_paths": ([P, ctypes.POINTER(i32)], ctypes.c_int),
        "tbe_table_backward_paths": ([P, ctypes.POINTER(i32)], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def declared_functions() -> List[str]:
    """Names of the functions include/tbe.h declares."""
    with open(HEADER_PATH) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(tbe_[a-z0-9_]+)\s*\(", text)))


def _check(rc: int, where: str):
    if rc != TBE_OK:
        if rc == TBE_ERR_CUDA:
            where = f"{where} (cudaError_t {load_library().tbe_last_cuda_error()})"
        raise TBEError(rc, where)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        # the current stream's handle without building a Stream object (3 us)
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()))
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _new(shape, dtype, device, stream, returned: bool = True) -> torch.Tensor:
    """Memory that a call allocates for its launches on ``stream``.  It belongs
    to that stream, so the allocator hands it on only behind them, and (what
    the call returns) waits for the current stream's use of it too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        at = _stream(stream).value
        stream = torch.cuda.ExternalStream(at, device=device) if at else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _index_dtype(indices: torch.Tensor, offsets: torch.Tensor) -> int:
    if indices.dtype != offsets.dtype or indices.dtype not in (torch.int32, torch.int64):
        raise ValueError("indices and offsets must share dtype int32 or int64")
    return TBE_I64 if indices.dtype == torch.int64 else TBE_I32


def tbe_strerror(code: int) -> str:
    try:
        return load_library().tbe_strerror(code).decode()
    except RuntimeError:
        return f"status {code}"


class Handle:
    """A created TBE handle.  Keeps the tables alive; ``close()`` (or garbage
    collection) calls tbe_destroy."""

    def __init__(self, ptr: ctypes.c_void_p, tables: Sequence[torch.Tensor], pooling: str):
        self._ptr = ptr
        self.tables = list(tables)
        self.pooling = pooling
        self.dims = [int(t.shape[1]) for t in tables]
        self.rows = [int(t.shape[0]) for t in tables]
        self.total_dim = sum(self.dims)
        self.total_rows = sum(self.rows)

    @property
    def ptr(self):
        if self._ptr is None:
            raise RuntimeError("handle already destroyed")
        return self._ptr

    def close(self):
        if self._ptr is not None and _lib is not None:
            _lib.tbe_destroy(self._ptr)
        self._ptr = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def tbe_create(tables: Sequence[torch.Tensor], pooling: str = "sum", flags: int = 0) -> Handle:
    """Tables: CUDA tensors [rows, dim] (fp32/fp16/bf16), updated in place by backward."""
    lib = load_library()
    arr = (_Table * len(tables))()
    for i, t in enumerate(tables):
        if t.dim() != 2 or t.dtype not in _DTYPES:
            raise ValueError("tables must be 2-D fp32/fp16/bf16 CUDA tensors")
        if not t.is_contiguous():
            raise ValueError("tables must be contiguous (row-major, rows packed)")
        arr[i] = _Table(t.shape[0], t.shape[1], _DTYPES[t.dtype], _ptr(t))
    out = ctypes.c_void_p()
    _check(lib.tbe_create(arr, len(tables), _POOL[pooling], flags, ctypes.byref(out)), "tbe_create")
    return Handle(out, tables, pooling)


def tbe_destroy(h: Handle):
    h.close()


def tbe_table_paths(h: Handle) -> List[str]:
    buf = (ctypes.c_int32 * len(h.tables))()
    _check(load_library().tbe_table_paths(h.ptr, buf), "tbe_table_paths")
    return [PATH_NAMES[int(x)] for x in buf]


def tbe_backward_paths(h: Handle) -> List[str]:
    """Per table, "dense" (tensor-core H^T . G) or "sorted"."""
    buf = (ctypes.c_int32 * len(h.tables))()
    _check(load_library().tbe_table_backward_paths(h.ptr, buf), "tbe_table_backward_paths")
    return ["dense" if int(x) else "sorted" for x in buf]


def tbe_forward(h: Handle, indices: torch.Tensor, offsets: torch.Tensor, batch_size: int,
                per_sample_weights: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    lib = load_library()
    if out is None:
        out = _new((batch_size, h.total_dim), torch.float32, offsets.device, stream)
    rc = lib.tbe_forward(h.ptr, _ptr(indices), _ptr(offsets), _index_dtype(indices, offsets),
                         indices.numel(), batch_size, _ptr(per_sample_weights), _ptr(out),
                         _stream(stream))
    _check(rc, "tbe_forward")
    return out


def tbe_per_sample_weight_grad(h: Handle, indices: torch.Tensor, offsets: torch.Tensor, batch_size: int,
                               grad_out: torch.Tensor, grad_weights: Optional[torch.Tensor] = None,
                               stream=None) -> torch.Tensor:
    """dL/dw_i for every lookup; call before the backward pass updates the rows."""
    lib = load_library()
    if grad_weights is None:
        grad_weights = _new((indices.numel(),), torch.float32, offsets.device, stream)
    rc = lib.tbe_per_sample_weight_grad(h.ptr, _ptr(indices), _ptr(offsets), _index_dtype(indices, offsets),
                                        indices.numel(), batch_size, _ptr(grad_out), _ptr(grad_weights),
                                        _stream(stream))
    _check(rc, "tbe_per_sample_weight_grad")
    return grad_weights


def tbe_backward_workspace_bytes(h: Handle, num_indices: int, batch_size: int) -> int:
    return int(load_library().tbe_backward_workspace_bytes(h.ptr, num_indices, batch_size))


def tbe_backward_workspace_layout(h: Handle, num_indices: int, batch_size: int) -> WorkspaceLayout:
    out = WorkspaceLayout()
    _check(load_library().tbe_backward_workspace_layout(h.ptr, num_indices, batch_size,
                                                        ctypes.byref(out)),
           "tbe_backward_workspace_layout")
    return out


def make_workspace(h: Handle, num_indices: int, batch_size: int, device=None, stream=None) -> torch.Tensor:
    """Workspace of a backward pass on ``stream`` (the current one by default)."""
    n = tbe_backward_workspace_bytes(h, num_indices, batch_size)
    return _new((n,), torch.uint8, device or h.tables[0].device, stream, False)


def tbe_backward_prepare(h: Handle, indices, offsets, batch_size: int, workspace: torch.Tensor,
                         per_sample_weights=None, stream=None):
    rc = load_library().tbe_backward_prepare(
        h.ptr, _ptr(indices), _ptr(offsets), _index_dtype(indices, offsets), indices.numel(),
        batch_size, _ptr(per_sample_weights), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "tbe_backward_prepare")


def tbe_forward_prepare(h: Handle, indices, offsets, batch_size: int, workspace: torch.Tensor,
                        per_sample_weights=None, out: Optional[torch.Tensor] = None, stream=None):
    """Forward pass and backward preparation of one batch, run side by side."""
    if out is None:
        out = _new((batch_size, h.total_dim), torch.float32, offsets.device, stream)
    rc = load_library().tbe_forward_prepare(
        h.ptr, _ptr(indices), _ptr(offsets), _index_dtype(indices, offsets), indices.numel(),
        batch_size, _ptr(per_sample_weights), _ptr(out), _ptr(workspace), workspace.numel(),
        _stream(stream))
    _check(rc, "tbe_forward_prepare")
    return out


def tbe_backward_apply(h: Handle, num_indices: int, batch_size: int, grad_out: torch.Tensor,
                       workspace: torch.Tensor, optimizer: str = "sgd", lr: float = 0.01,
                       eps: float = 0.0, state: Optional[torch.Tensor] = None, stream=None):
    kind = TBE_OPT_SGD if optimizer == "sgd" else TBE_OPT_ROWWISE_ADAGRAD
    opt = _Optimizer(kind, lr, eps, _ptr(state))
    rc = load_library().tbe_backward_apply(h.ptr, num_indices, batch_size, _ptr(grad_out),
                                           ctypes.byref(opt), _ptr(workspace), workspace.numel(),
                                           _stream(stream))
    _check(rc, "tbe_backward_apply")


def tbe_backward_sgd(h: Handle, indices, offsets, batch_size: int, grad_out, lr: float,
                     workspace: torch.Tensor, per_sample_weights=None, stream=None):
    rc = load_library().tbe_backward_sgd(
        h.ptr, _ptr(indices), _ptr(offsets), _index_dtype(indices, offsets), indices.numel(),
        batch_size, _ptr(per_sample_weights), _ptr(grad_out), lr, _ptr(workspace),
        workspace.numel(), _stream(stream))
    _check(rc, "tbe_backward_sgd")


def tbe_backward_rowwise_adagrad(h: Handle, indices, offsets, batch_size: int, grad_out,
                                 state: torch.Tensor, lr: float, eps: float,
                                 workspace: torch.Tensor, per_sample_weights=None, stream=None):
    rc = load_library().tbe_backward_rowwise_adagrad(
        h.ptr, _ptr(indices), _ptr(offsets), _index_dtype(indices, offsets), indices.numel(),
        batch_size, _ptr(per_sample_weights), _ptr(grad_out), _ptr(state), lr, eps,
        _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "tbe_backward_rowwise_adagrad")


def tbe_backward_sgd_noalloc(h: Handle, indices, offsets, batch_size: int, grad_out, lr: float,
                             per_sample_weights=None, stream=None):
    """tbe_backward_sgd with the library's static 32 MiB workspace: for callers
    that cannot allocate device memory for a workspace (see include/tbe.h)."""
    rc = load_library().tbe_backward_sgd_noalloc(
        h.ptr, _ptr(indices), _ptr(offsets), _index_dtype(indices, offsets), indices.numel(),
        batch_size, _ptr(per_sample_weights), _ptr(grad_out), lr, _stream(stream))
    _check(rc, "tbe_backward_sgd_noalloc")


def tbe_get_error(h: Handle, stream=None) -> int:
    return int(load_library().tbe_get_error(h.ptr, _stream(stream)))


# ------------------------------------------------- attention over histories


class AttentionHandle:
    """A created attention handle; ``close()`` (or garbage collection) calls
    tbe_attention_destroy."""

    def __init__(self, ptr: ctypes.c_void_p, heads: int, kv_heads: int, head_dim: int, dtype: torch.dtype,
                 buckets: int):
        self._ptr = ptr
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.dtype, self.buckets = dtype, buckets

    @property
    def ptr(self):
        if self._ptr is None:
            raise RuntimeError("handle already destroyed")
        return self._ptr

    def close(self):
        if self._ptr is not None and _lib is not None:
            _lib.tbe_attention_destroy(self._ptr)
        self._ptr = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def tbe_relative_buckets(num_buckets: int, max_distance: int) -> List[int]:
    """First distance of each bucket of a learned relative position bias: one
    distance per bucket in the first half, then growing by a constant factor;
    distances of max_distance and more share the last bucket."""
    if num_buckets < 1 or max_distance < num_buckets:
        raise ValueError("needs 1 <= num_buckets <= max_distance")
    single = max(1, num_buckets // 2)
    starts = list(range(min(single, num_buckets)))
    wide = num_buckets - single
    for i in range(wide):
        at = max_distance if i == wide - 1 else math.ceil(
            single * (max_distance / single) ** (i / (wide - 1)) - 1e-9)
        starts.append(max(starts[-1] + 1, at))
    return starts


def tbe_attention_create(heads: int, kv_heads: int, head_dim: int, dtype: torch.dtype, window: int = 0,
                         sinks: int = 0, bucket_starts: Optional[Sequence[int]] = None,
                         scale: Optional[float] = None) -> AttentionHandle:
    """Attention over ragged histories: each token sees the ``window`` newest
    tokens up to itself (0: all) and the first ``sinks``; ``bucket_starts``
    (see tbe_relative_buckets) adds a learned bias by distance; ``scale``
    defaults to head_dim ** -0.5."""
    if dtype not in _DTYPES:
        raise ValueError("dtype must be fp32, fp16 or bf16")
    firsts = [] if bucket_starts is None else [int(x) for x in bucket_starts]
    for x in (heads, kv_heads, head_dim, window, sinks, *firsts):
        if not -2 ** 31 <= x < 2 ** 31:  # a C int32 field would keep its low bits
            raise ValueError(f"{x} is outside int32")
    lib = load_library()
    n = len(firsts)
    starts = (ctypes.c_int32 * max(n, 1))(*firsts)
    cfg = _AttentionConfig(_DTYPES[dtype], heads, kv_heads, head_dim, window, sinks,
                           head_dim ** -0.5 if scale is None else scale, n, starts)
    out = ctypes.c_void_p()
    _check(lib.tbe_attention_create(ctypes.byref(cfg), ctypes.byref(out)), "tbe_attention_create")
    return AttentionHandle(out, heads, kv_heads, head_dim, dtype, n)


def tbe_attention_destroy(h: AttentionHandle):
    h.close()


# The calls below are made once per request by a serving loop: their checks
# use few Python objects (addresses as ints, torch.Size compared as it is).

def _refuse(name: str, t: torch.Tensor, shape, dtype) -> None:
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected {list(shape)}, got {list(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    raise ValueError(f"{name}: the last dimension must be contiguous")


def _rows(h: AttentionHandle, t: torch.Tensor, tokens: int, heads: int, name: str) -> _Rows:
    d = h.head_dim
    if t.shape != (tokens, heads, d) or t.dtype is not h.dtype or not t.is_cuda:
        _refuse(name, t, (tokens, heads, d), h.dtype)
    s0, s1, s2 = t.stride()
    if s2 != 1 and d > 1:
        _refuse(name, t, t.shape, t.dtype)
    return _Rows(t.data_ptr(), s0, s1)


def _pages(h: AttentionHandle, t: torch.Tensor, shape, name: str) -> _Pages:
    if t.shape != shape or t.dtype is not h.dtype or not t.is_cuda:
        _refuse(name, t, shape, h.dtype)
    s0, s1, s2, s3 = t.stride()
    if s3 != 1 and h.head_dim > 1:
        _refuse(name, t, t.shape, t.dtype)
    return _Pages(t.data_ptr(), s0, s1, s2)


def _packed(t: torch.Tensor, shape, dtype, name: str) -> int:
    """Address of a contiguous CUDA tensor of this shape and type."""
    if t.shape != shape or t.dtype is not dtype or not t.is_cuda:
        _refuse(name, t, shape, dtype)
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return t.data_ptr()


def _space(t: torch.Tensor) -> int:
    if not t.is_cuda or not t.is_contiguous() or t.dtype is not torch.uint8:
        raise ValueError("workspace: expected a contiguous CUDA tensor of bytes")
    at = t.data_ptr()
    if at % 16:
        raise ValueError("workspace: expected memory on a 16-byte boundary")
    return at


def _bias(h: AttentionHandle, bias: Optional[torch.Tensor]):
    if (bias is None) != (h.buckets == 0):
        raise ValueError("bias must be given exactly where the handle has buckets")
    return None if bias is None else _packed(bias, (h.buckets, h.heads), h.dtype, "bias")


def _offsets(offsets: torch.Tensor):
    """(address, index type, histories) of B+1 offsets."""
    if offsets.dim() != 1 or offsets.shape[0] < 1 or offsets.dtype not in (torch.int32, torch.int64):
        raise ValueError("offsets must be a 1-D int32 or int64 tensor of B+1 entries")
    at = _packed(offsets, offsets.shape, offsets.dtype, "offsets")
    return at, TBE_I64 if offsets.dtype is torch.int64 else TBE_I32, offsets.shape[0] - 1


def tbe_attention_workspace_bytes(h: AttentionHandle, num_tokens: int, batch_size: int,
                                  backward: bool = False) -> int:
    return int(load_library().tbe_attention_workspace_bytes(h.ptr, num_tokens, batch_size, int(backward)))


def make_attention_workspace(h: AttentionHandle, num_tokens: int, batch_size: int, backward: bool = False,
                             device=None, stream=None) -> torch.Tensor:
    """Workspace of forward calls (``backward``: of both) up to this size, on
    ``stream`` (the current one by default)."""
    n = tbe_attention_workspace_bytes(h, num_tokens, batch_size, backward)
    if n == 0:
        raise TBEError(TBE_ERR_UNSUPPORTED, "tbe_attention_workspace_bytes")
    return _new((n,), torch.uint8, device or "cuda", stream, False)


def tbe_attention_forward(h: AttentionHandle, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                          offsets: torch.Tensor, bias: Optional[torch.Tensor] = None,
                          out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None):
    """q [N, H, D], k and v [N, Hk, D] of the batch's histories (strided rows
    are fine), offsets [B+1]; returns (out [N, H, D], lse [H, N])."""
    n, heads = q.shape[0], h.heads
    rq, rk, rv = _rows(h, q, n, heads, "q"), _rows(h, k, n, h.kv_heads, "k"), _rows(h, v, n, h.kv_heads, "v")
    po, it, b = _offsets(offsets)
    shape = (n, heads, h.head_dim)
    if out is None:
        out = _new(shape, h.dtype, q.device, stream)
    if lse is None:
        lse = _new((heads, n), torch.float32, q.device, stream)
    if workspace is None:
        workspace = make_attention_workspace(h, n, b, False, q.device, stream)
    rc = load_library().tbe_attention_forward(
        h.ptr, rq, rk, rv, _bias(h, bias), po, it, n, b, _packed(out, shape, h.dtype, "out"),
        _packed(lse, (heads, n), torch.float32, "lse"), _space(workspace), workspace.numel(), _stream(stream))
    _check(rc, "tbe_attention_forward")
    return out, lse


def tbe_attention_backward(h: AttentionHandle, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                           offsets: torch.Tensor, out: torch.Tensor, lse: torch.Tensor, grad_out: torch.Tensor,
                           bias: Optional[torch.Tensor] = None, grad_q: Optional[torch.Tensor] = None,
                           grad_k: Optional[torch.Tensor] = None, grad_v: Optional[torch.Tensor] = None,
                           grad_bias: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                           stream=None):
    """Gradients (grad_q, grad_k, grad_v, grad_bias) from a forward call's out
    and lse and the upstream gradient; grad_bias is None without buckets."""
    n, heads, kv, d, dt = q.shape[0], h.heads, h.kv_heads, h.head_dim, h.dtype
    rq, rk, rv = _rows(h, q, n, heads, "q"), _rows(h, k, n, kv, "k"), _rows(h, v, n, kv, "v")
    rg = _rows(h, grad_out, n, heads, "grad_out")
    po, it, b = _offsets(offsets)
    if grad_q is None:
        grad_q = _new((n, heads, d), dt, q.device, stream)
    if grad_k is None:
        grad_k = _new((n, kv, d), dt, q.device, stream)
    if grad_v is None:
        grad_v = _new((n, kv, d), dt, q.device, stream)
    pb = None
    if h.buckets:
        if grad_bias is None:
            grad_bias = _new((h.buckets, heads), dt, q.device, stream)
        pb = _packed(grad_bias, (h.buckets, heads), dt, "grad_bias")
    elif grad_bias is not None:
        raise ValueError("grad_bias without buckets")
    if workspace is None:
        workspace = make_attention_workspace(h, n, b, True, q.device, stream)
    rc = load_library().tbe_attention_backward(
        h.ptr, rq, rk, rv, _bias(h, bias), po, it, n, b, _packed(out, (n, heads, d), dt, "out"),
        _packed(lse, (heads, n), torch.float32, "lse"), rg, _packed(grad_q, (n, heads, d), dt, "grad_q"),
        _packed(grad_k, (n, kv, d), dt, "grad_k"), _packed(grad_v, (n, kv, d), dt, "grad_v"), pb, _space(workspace),
        workspace.numel(), _stream(stream))
    _check(rc, "tbe_attention_backward")
    return grad_q, grad_k, grad_v, grad_bias


def _cache(h: AttentionHandle, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor, b: int):
    if k_pages.dim() != 4 or block_table.dim() != 2:
        raise ValueError("pages must be [pages, page size, Hk, D], block_table [B, width]")
    pages, size = k_pages.shape[0], k_pages.shape[1]
    width = block_table.shape[1]
    shape = (pages, size, h.kv_heads, h.head_dim)
    return (_pages(h, k_pages, shape, "k_pages"), _pages(h, v_pages, shape, "v_pages"), pages, size,
            _packed(block_table, (b, width), torch.int32, "block_table"), width)


def tbe_attention_append(h: AttentionHandle, k: torch.Tensor, v: torch.Tensor, offsets: torch.Tensor,
                         before: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                         block_table: torch.Tensor, stream=None):
    """Writes new tokens' keys and values ([N, Hk, D], ragged by offsets) into
    the paged cache ([pages, page size, Hk, D]) behind the ``before`` tokens
    each history holds already; block_table [B, width] names its pages."""
    n = k.shape[0]
    rk, rv = _rows(h, k, n, h.kv_heads, "k"), _rows(h, v, n, h.kv_heads, "v")
    po, it, b = _offsets(offsets)
    kp, vp, pages, size, table, width = _cache(h, k_pages, v_pages, block_table, b)
    rc = load_library().tbe_attention_append(
        h.ptr, rk, rv, po, it, n, b, _packed(before, (b,), torch.int32, "before"), kp, vp, pages, size, table, width,
        _stream(stream))
    _check(rc, "tbe_attention_append")


def tbe_attention_decode_workspace_bytes(h: AttentionHandle, batch_size: int, max_length: int) -> int:
    return int(load_library().tbe_attention_decode_workspace_bytes(h.ptr, batch_size, max_length))


def make_attention_decode_workspace(h: AttentionHandle, batch_size: int, max_length: int,
                                    device=None, stream=None) -> torch.Tensor:
    """Workspace of decode calls of up to this many histories and tokens each,
    on ``stream`` (the current one by default)."""
    n = tbe_attention_decode_workspace_bytes(h, batch_size, max_length)
    if n == 0:
        raise TBEError(TBE_ERR_UNSUPPORTED, "tbe_attention_decode_workspace_bytes")
    return _new((n,), torch.uint8, device or "cuda", stream, False)


def tbe_attention_decode(h: AttentionHandle, q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                         block_table: torch.Tensor, lengths: torch.Tensor, bias: Optional[torch.Tensor] = None,
                         max_length: Optional[int] = None, out: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of each history's newest token (q [B, H, D]) over its paged
    cache of ``lengths`` tokens (the newest included); max_length, an upper
    bound of them, is the block table's room if it is not given or 0."""
    b, shape = q.shape[0], q.shape
    rq = _rows(h, q, b, h.heads, "q")
    kp, vp, pages, size, table, width = _cache(h, k_pages, v_pages, block_table, b)
    most = int(max_length or 0) or width * size
    if out is None:
        out = _new(shape, h.dtype, q.device, stream)
    if workspace is None:
        workspace = make_attention_decode_workspace(h, b, most, q.device, stream)
    rc = load_library().tbe_attention_decode(
        h.ptr, rq, kp, vp, pages, size, table, width, _packed(lengths, (b,), torch.int32, "lengths"), b, most,
        _bias(h, bias), _packed(out, shape, h.dtype, "out"), _space(workspace), workspace.numel(), _stream(stream))
    _check(rc, "tbe_attention_decode")
    return out


def tbe_attention_get_error(h: AttentionHandle, stream=None) -> int:
    return int(load_library().tbe_attention_get_error(h.ptr, _stream(stream)))


# ------------------------------------------------------ layer normalisation


class LayerNormHandle:
    """A created layer norm handle; ``close()`` (or garbage collection) calls
    tbe_layer_norm_destroy."""

    def __init__(self, ptr: ctypes.c_void_p, dim: int, dtype: torch.dtype, weight: bool, bias: bool):
        self._ptr = ptr
        self.dim, self.dtype, self.weight, self.bias = dim, dtype, weight, bias
        self.device = torch.cuda.current_device()

    @property
    def ptr(self):
        if self._ptr is None:
            raise RuntimeError("handle already destroyed")
        return self._ptr

    def close(self):
        if self._ptr is not None and _lib is not None:
            _lib.tbe_layer_norm_destroy(self._ptr)
        self._ptr = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def tbe_layer_norm_create(dim: int, dtype: torch.dtype, eps: float = 1e-5, weight: bool = True,
                          bias: bool = True) -> LayerNormHandle:
    """Layer norm of rows of ``dim`` elements; ``weight`` and ``bias`` say
    whether it has them."""
    if dtype not in _DTYPES:
        raise ValueError("dtype must be fp32, fp16 or bf16")
    if not -2 ** 31 <= dim < 2 ** 31:  # a C int32 field would keep its low bits
        raise ValueError(f"{dim} is outside int32")
    cfg = _LayerNormConfig(_DTYPES[dtype], dim, eps, int(bool(weight)), int(bool(bias)))
    out = ctypes.c_void_p()
    _check(load_library().tbe_layer_norm_create(ctypes.byref(cfg), ctypes.byref(out)), "tbe_layer_norm_create")
    return LayerNormHandle(out, dim, dtype, bool(weight), bool(bias))


def tbe_layer_norm_destroy(h: LayerNormHandle):
    h.close()


def _on_device(h, *tensors: Optional[torch.Tensor]) -> None:
    """Refuses tensors of another device than the handle's: the launches go to
    that one."""
    for t in tensors:
        if t is not None and t.get_device() != h.device:
            raise ValueError(f"expected tensors on cuda:{h.device}, got {t.device}")


def _matrix(t: torch.Tensor, rows: int, dim: int, dtype, name: str):
    """(address, row stride) of a [rows, dim] CUDA tensor with packed elements."""
    if t.shape != (rows, dim) or t.dtype is not dtype or not t.is_cuda:
        _refuse(name, t, (rows, dim), dtype)
    s0, s1 = t.stride()
    if s1 != 1 and dim > 1:
        _refuse(name, t, t.shape, t.dtype)
    return t.data_ptr(), s0


def _result(t: Optional[torch.Tensor], shape, dtype, like: torch.Tensor, stream, name: str):
    """(tensor, address) of a result: the caller's, or memory of the call's own
    beside ``like``."""
    if t is None:
        t = _new(shape, dtype, like.device, stream)
        return t, t.data_ptr()
    return t, _packed(t, shape, dtype, name)


def _param(t: Optional[torch.Tensor], has: bool, dim: int, dtype, name: str):
    if (t is not None) != has:
        raise ValueError(f"{name} must be given exactly where the handle has one")
    return None if t is None else _packed(t, (dim,), dtype, name)


def tbe_layer_norm_forward(h: LayerNormHandle, x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                           bias: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                           out: Optional[torch.Tensor] = None, total: Optional[torch.Tensor] = None,
                           stats: Optional[torch.Tensor] = None, stream=None):
    """x [N, D] and residual [N, D] (strided rows are fine); returns (out,
    total, stats): the normalised rows, the kept stream x + residual (x itself
    without a residual, None where ``out`` has taken its place: there is nothing
    left for a backward call) and fp32 [2, N] of the rows' mean and 1 / deviation."""
    if x.dim() != 2:
        raise ValueError("x must be [N, D]")
    n, d, dt = x.shape[0], h.dim, h.dtype
    px, sx = _matrix(x, n, d, dt, "x")
    pr, sr, pt = None, 0, None
    pw, pb = _param(weight, h.weight, d, dt, "weight"), _param(bias, h.bias, d, dt, "bias")
    _on_device(h, x, residual, weight, bias, out, total, stats)
    out, po = _result(out, (n, d), dt, x, stream, "out")
    stats, ps = _result(stats, (2, n), torch.float32, x, stream, "stats")
    if residual is not None:
        pr, sr = _matrix(residual, n, d, dt, "residual")
        total, pt = _result(total, (n, d), dt, x, stream, "total")
    elif total is not None:
        raise ValueError("total without residual")
    rc = load_library().tbe_layer_norm_forward(h.ptr, px, sx, pr, sr, pw, pb, n, po, pt, ps, _stream(stream))
    _check(rc, "tbe_layer_norm_forward")
    if residual is None:
        total = None if n > 0 and po == px else x
    return out, total, stats


def tbe_layer_norm_workspace_bytes(h: LayerNormHandle, num_rows: int) -> int:
    return int(load_library().tbe_layer_norm_workspace_bytes(h.ptr, num_rows))


def make_layer_norm_workspace(h: LayerNormHandle, num_rows: int, device=None, stream=None) -> torch.Tensor:
    """Workspace of backward calls of up to this many rows, on ``stream`` (the
    current one by default)."""
    n = tbe_layer_norm_workspace_bytes(h, num_rows)
    if n == 0:
        raise TBEError(TBE_ERR_UNSUPPORTED, "tbe_layer_norm_workspace_bytes")
    return _new((n,), torch.uint8, device or "cuda", stream, False)


def tbe_layer_norm_backward(h: LayerNormHandle, total: torch.Tensor, stats: torch.Tensor, grad_out: torch.Tensor,
                            weight: Optional[torch.Tensor] = None, grad_total: Optional[torch.Tensor] = None,
                            grad_x: Optional[torch.Tensor] = None, grad_weight: Optional[torch.Tensor] = None,
                            grad_bias: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                            stream=None):
    """Gradients (grad_x, grad_weight, grad_bias) from a forward call's total
    and stats and the upstream gradients of its out and (optionally) its total;
    grad_x is the residual's gradient too.  What the handle has no parameter
    for is None."""
    if total is None or total.dim() != 2:
        raise ValueError("total must be [N, D]")
    n, d, dt = total.shape[0], h.dim, h.dtype
    pt, st = _matrix(total, n, d, dt, "total")
    pg, sg = _matrix(grad_out, n, d, dt, "grad_out")
    pu, su = (None, 0) if grad_total is None else _matrix(grad_total, n, d, dt, "grad_total")
    pw, ps = _param(weight, h.weight, d, dt, "weight"), _packed(stats, (2, n), torch.float32, "stats")
    _on_device(h, total, stats, grad_out, grad_total, weight, grad_x, grad_weight, grad_bias, workspace)
    px = pgw = pgb = None
    grad_x, px = _result(grad_x, (n, d), dt, total, stream, "grad_x")
    if h.weight:
        grad_weight, pgw = _result(grad_weight, (d,), dt, total, stream, "grad_weight")
    elif grad_weight is not None:
        raise ValueError("grad_weight without weight")
    if h.bias:
        grad_bias, pgb = _result(grad_bias, (d,), dt, total, stream, "grad_bias")
    elif grad_bias is not None:
        raise ValueError("grad_bias without bias")
    if workspace is None:
        workspace = make_layer_norm_workspace(h, n, total.device, stream)
    rc = load_library().tbe_layer_norm_backward(h.ptr, pt, st, ps, pg, sg, pu, su, pw, n, px, pgw, pgb,
                                                _space(workspace), workspace.numel(), _stream(stream))
    _check(rc, "tbe_layer_norm_backward")
    return grad_x, grad_weight, grad_bias


# ---------------------------------------- softmax loss over a table of items


class SoftmaxLossHandle:
    """A created loss handle; ``close()`` (or garbage collection) calls
    tbe_softmax_loss_destroy."""

    def __init__(self, ptr: ctypes.c_void_p, dim: int, dtype: torch.dtype):
        self._ptr = ptr
        self.dim, self.dtype = dim, dtype
        self.device = torch.cuda.current_device()

    @property
    def ptr(self):
        if self._ptr is None:
            raise RuntimeError("handle already destroyed")
        return self._ptr

    def close(self):
        if self._ptr is not None and _lib is not None:
            _lib.tbe_softmax_loss_destroy(self._ptr)
        self._ptr = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def tbe_softmax_loss_create(dim: int, dtype: torch.dtype, scale: float = 1.0) -> SoftmaxLossHandle:
    """Softmax cross entropy of rows of ``dim`` elements over a table of items;
    logits are ``scale`` times the products (an inverse temperature)."""
    if dtype not in _DTYPES:
        raise ValueError("dtype must be fp32, fp16 or bf16")
    if not -2 ** 31 <= dim < 2 ** 31:  # a C int32 field would keep its low bits
        raise ValueError(f"{dim} is outside int32")
    cfg = _SoftmaxLossConfig(_DTYPES[dtype], dim, scale)
    out = ctypes.c_void_p()
    _check(load_library().tbe_softmax_loss_create(ctypes.byref(cfg), ctypes.byref(out)), "tbe_softmax_loss_create")
    return SoftmaxLossHandle(out, dim, dtype)


def tbe_softmax_loss_destroy(h: SoftmaxLossHandle):
    h.close()


def tbe_softmax_loss_workspace_bytes(h: SoftmaxLossHandle, num_rows: int, num_items: int,
                                     backward: bool = False) -> int:
    return int(load_library().tbe_softmax_loss_workspace_bytes(h.ptr, num_rows, num_items, int(backward)))


def make_softmax_loss_workspace(h: SoftmaxLossHandle, num_rows: int, num_items: int, backward: bool = False,
                                device=None, stream=None) -> torch.Tensor:
    """Workspace of forward calls (``backward``: of both) of up to this many
    rows and items, on ``stream`` (the current one by default)."""
    n = tbe_softmax_loss_workspace_bytes(h, num_rows, num_items, backward)
    if n == 0:
        raise TBEError(TBE_ERR_UNSUPPORTED, "tbe_softmax_loss_workspace_bytes")
    return _new((n,), torch.uint8, device or "cuda", stream, False)


def _loss_operands(h: SoftmaxLossHandle, x: torch.Tensor, table: torch.Tensor, targets: torch.Tensor):
    """(x, its stride, table, its stride, targets, their type, rows, items)."""
    if x.dim() != 2 or table.dim() != 2:
        raise ValueError("x must be [N, D], table [V, D]")
    if targets.dtype not in (torch.int32, torch.int64):
        raise ValueError("targets must be int32 or int64")
    n, v = x.shape[0], table.shape[0]
    return (*_matrix(x, n, h.dim, h.dtype, "x"), *_matrix(table, v, h.dim, h.dtype, "table"),
            _packed(targets, (n,), targets.dtype, "targets"), TBE_I64 if targets.dtype is torch.int64 else TBE_I32,
            n, v)


def tbe_softmax_loss_forward(h: SoftmaxLossHandle, x: torch.Tensor, table: torch.Tensor, targets: torch.Tensor,
                             loss: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                             workspace: Optional[torch.Tensor] = None, stream=None):
    """x [N, D] states and table [V, D] (strided rows are fine), targets [N]
    (the item of each row; negative: the row is left out); returns (loss, lse),
    both fp32 [N]."""
    ops = _loss_operands(h, x, table, targets)
    n, v = ops[-2:]
    _on_device(h, x, table, targets, loss, lse, workspace)
    loss, po = _result(loss, (n,), torch.float32, x, stream, "loss")
    lse, pl = _result(lse, (n,), torch.float32, x, stream, "lse")
    if workspace is None:
        workspace = make_softmax_loss_workspace(h, n, v, False, x.device, stream)
    rc = load_library().tbe_softmax_loss_forward(h.ptr, *ops, po, pl, _space(workspace), workspace.numel(),
                                                 _stream(stream))
    _check(rc, "tbe_softmax_loss_forward")
    return loss, lse


def tbe_softmax_loss_backward(h: SoftmaxLossHandle, x: torch.Tensor, table: torch.Tensor, targets: torch.Tensor,
                              lse: torch.Tensor, grad_loss: torch.Tensor, grad_x: Optional[torch.Tensor] = None,
                              grad_table: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                              want=(True, True), stream=None):
    """Gradients (grad_x [N, D], grad_table [V, D]) from a forward call's lse and
    the upstream gradient of its losses (fp32 [N]); ``want`` says which of them
    are computed (the other is None)."""
    ops = _loss_operands(h, x, table, targets)
    n, v = ops[-2:]
    pl, pg = _packed(lse, (n,), torch.float32, "lse"), _packed(grad_loss, (n,), torch.float32, "grad_loss")
    _on_device(h, x, table, targets, lse, grad_loss, grad_x, grad_table, workspace)
    px = pt = None
    if want[0] or grad_x is not None:
        grad_x, px = _result(grad_x, (n, h.dim), h.dtype, x, stream, "grad_x")
    if want[1] or grad_table is not None:
        grad_table, pt = _result(grad_table, (v, h.dim), h.dtype, x, stream, "grad_table")
    if workspace is None:
        workspace = make_softmax_loss_workspace(h, n, v, True, x.device, stream)
    rc = load_library().tbe_softmax_loss_backward(h.ptr, *ops, pl, pg, px, pt, _space(workspace), workspace.numel(),
                                                  _stream(stream))
    _check(rc, "tbe_softmax_loss_backward")
    return grad_x, grad_table


def tbe_softmax_loss_get_error(h: SoftmaxLossHandle, stream=None) -> int:
    return int(load_library().tbe_softmax_loss_get_error(h.ptr, _stream(stream)))


__all__ = [n for n in dir() if n.startswith("tbe_") or n.startswith("TBE_")] + [
    "Handle", "TBEError", "WorkspaceLayout", "load_library", "declared_functions",
    "make_workspace", "library_path", "AttentionHandle", "make_attention_workspace",
    "make_attention_decode_workspace", "LayerNormHandle", "make_layer_norm_workspace", "SoftmaxLossHandle",
    "make_softmax_loss_workspace"]
