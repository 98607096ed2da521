"""Python binding of the GB300 k-means library (``include/kmeans_gb300.h``).

Argument marshalling only: every function checks tensor types, shapes and
devices, passes raw device pointers, sizes and the current CUDA stream to the
C ABI of ``libkmeans_gb300.so``, and raises ``KMeansError`` on a non-zero
status.  All arithmetic runs in the library's CUDA kernels.  PyTorch supplies
device memory (outputs and the workspace when the caller passes none) and
streams.  There is no CPU path: without the built library every call fails.

Names follow the C ABI: ``kmeans_assign``, ``kmeans_assign_ffma``,
``kmeans_update``, ``kmeans_lloyd_iter``, ``kmeanspp_init``,
``kmeans_workspace_bytes``, ``kmeans_device_status``, ``kmeans_status_string``,
and the shard entry points (``kmeans_lloyd_iter_partial``,
``kmeans_reduce_partials``, ``kmeanspp_shard_*``) that ``sharded.py`` drives
across processes.  ``kmeans_route*`` and ``kmeans_linear*`` are the expert
routing and the experts' products that ``experts.py`` makes a layer of;
``kmeans_gate``, ``kmeans_layernorm`` and ``kmeans_cross_entropy`` (each with
its ``_grad``) stand around them.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libkmeans_gb300.so")

KMEANS_OK = 0
KMEANS_ERR_INVALID_ARG = 1
KMEANS_ERR_UNSUPPORTED = 2
KMEANS_ERR_WORKSPACE = 3
KMEANS_ERR_CUDA = 4
KMEANS_ERR_DEVICE_TIMEOUT = 5
KMEANS_ERR_DEVICE_LABEL = 6
KMEANS_ERR_SCRATCH_LIMIT = 7
KMEANS_ERR_DEVICE_EXCHANGE = 8
NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024

OP_ASSIGN = 0
OP_ASSIGN_FFMA = 1
OP_UPDATE = 2
OP_LLOYD = 3
OP_KMEANSPP = 4
OP_FIT = 5
OP_ASSIGN_3XTF32 = 6
OP_LLOYD_FUSED = 7
OP_RELOCATE = 8
OP_KMEANSPP_SHARD = 9
OP_LLOYD_PARTIAL = 10
OP_UPDATE_PARTIAL = 11

# kmeans_linear_workspace_bytes
OP_LINEAR = 0
OP_LINEAR_GRAD = 1
# kmeans_cross_entropy_workspace_bytes
OP_CROSS_ENTROPY = 0
OP_CROSS_ENTROPY_GRAD = 1

F32 = 0
F16 = 1
BF16 = 2
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
ROUTE_MAX_EXPERTS = 4096
ROUTE_MAX_TOPK = 32
ROUTE_MAX_WIDTH = 16000000
LINEAR_MAX_EXPERTS = 1024
LINEAR_MAX_SIZE = 2 ** 31 - 256
GATE_SCORES = {"softmax": 0, "sigmoid": 1}
GATE_MAX_GROUPS = 32
CROSS_ENTROPY_MAX_WIDTH = 32768

INIT_GIVEN = 0
INIT_KMEANSPP = 1
FIT_RELOCATE_EMPTY = 0x100

KERNEL_ASSIGN_TC = 0
KERNEL_UPDATE_MEAN = 1
KERNEL_KMEANSPP_DIST = 2
TRACE_MAX_CAPACITY = 65536
HOST_MAX_SLICES = 64
HOST_OVERLAP_PREVIOUS = 1
HOST_READBACK_ON_COPY_STREAM = 2
# Features per slice of the k-means++ distance pass: each pass writes one
# float2 partial sum per (slice, trial, sample), ceil(d / 4096) slices.
KPP_SLICE_FEATURES = 4096

# Every symbol the header declares (the ABI test checks the library exports them).
EXPORTS = (
    "kmeans_workspace_bytes", "kmeans_assign", "kmeans_assign_ffma", "kmeans_update",
    "kmeans_lloyd_iter", "kmeanspp_init", "kmeans_device_status", "kmeans_status_string",
    "kmeans_build_info", "kmeans_assign_noalloc", "kmeans_trace_start", "kmeans_trace_read",
    "kmeans_trace_stop", "kmeans_lloyd_iter_host", "kmeans_fit", "kmeans_assign_3xtf32",
    "kmeans_lloyd_iter_fused", "kmeans_relocate_empty", "kmeans_update_partial", "kmeans_lloyd_iter_partial",
    "kmeans_reduce_partials", "kmeanspp_shard_exchange_bytes", "kmeanspp_shard_first", "kmeanspp_shard_pick",
    "kmeanspp_shard_dist", "kmeanspp_shard_commit", "kmeanspp_rows_read",
    "kmeans_route_workspace_bytes", "kmeans_route", "kmeans_route_gather", "kmeans_route_combine",
    "kmeans_route_combine_grad", "kmeans_linear_workspace_bytes", "kmeans_linear", "kmeans_linear_grad",
    "kmeans_gate", "kmeans_gate_grad", "kmeans_layernorm_workspace_bytes", "kmeans_layernorm",
    "kmeans_layernorm_grad", "kmeans_cross_entropy_workspace_bytes", "kmeans_cross_entropy",
    "kmeans_cross_entropy_grad",
)

_lock = threading.Lock()
_lib = None


class KMeansError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {kmeans_status_string(status)} (status {status})")


def load(path: str | None = None):
    """Load the library once; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"{p} is missing: build it with `python -m distance_argmin_gb300.build`"
                               " (the library has no CPU fallback)")
        lib = ctypes.CDLL(p)
        P, I64, U64, SZ, INT = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint64, ctypes.c_size_t,
                                ctypes.c_int)
        lib.kmeans_workspace_bytes.argtypes = [INT, I64, I64, I64]
        lib.kmeans_workspace_bytes.restype = SZ
        assign_sig = [P, P, I64, I64, I64, P, P, P, P, SZ, U64, P]
        lib.kmeans_assign.argtypes = assign_sig
        lib.kmeans_assign.restype = INT
        lib.kmeans_assign_3xtf32.argtypes = assign_sig
        lib.kmeans_assign_3xtf32.restype = INT
        lib.kmeans_assign_ffma.argtypes = assign_sig
        lib.kmeans_assign_ffma.restype = INT
        lib.kmeans_assign_noalloc.argtypes = [P, P, I64, I64, I64, P, P, P, U64, P]
        lib.kmeans_assign_noalloc.restype = INT
        lib.kmeans_update.argtypes = [P, P, P, P, P, I64, I64, I64, P, SZ, U64, P]
        lib.kmeans_update.restype = INT
        lib.kmeans_lloyd_iter.argtypes = [P, P, P, P, P, P, P, I64, I64, I64, P, SZ, U64, P]
        lib.kmeans_lloyd_iter_fused.argtypes = lib.kmeans_lloyd_iter.argtypes
        lib.kmeans_lloyd_iter_fused.restype = INT
        lib.kmeans_lloyd_iter.restype = INT
        lib.kmeanspp_init.argtypes = [P, I64, I64, I64, INT, U64, P, P, P, SZ, P]
        lib.kmeanspp_init.restype = INT
        lib.kmeans_device_status.argtypes = [P, P]
        lib.kmeans_device_status.restype = INT
        lib.kmeanspp_rows_read.argtypes = [P, P, ctypes.POINTER(I64)]
        lib.kmeanspp_rows_read.restype = INT
        lib.kmeans_status_string.argtypes = [INT]
        lib.kmeans_status_string.restype = ctypes.c_char_p
        lib.kmeans_build_info.argtypes = []
        lib.kmeans_build_info.restype = ctypes.c_char_p
        lib.kmeans_trace_start.argtypes = [INT]
        lib.kmeans_trace_start.restype = INT
        lib.kmeans_trace_read.argtypes = [INT, P, P, P]
        lib.kmeans_trace_read.restype = INT
        lib.kmeans_lloyd_iter_host.argtypes = [P, P, P, P, P, P, P, P, P, P, P, P, I64, I64, I64, INT, INT, P, SZ, P,
                                               P]
        lib.kmeans_lloyd_iter_host.restype = INT
        lib.kmeans_fit.argtypes = [P, P, P, P, P, I64, I64, I64, INT, U64, INT, ctypes.c_double, P, P, P, SZ, P]
        lib.kmeans_fit.restype = INT
        lib.kmeans_relocate_empty.argtypes = [P, P, I64, I64, P, SZ, P]
        lib.kmeans_relocate_empty.restype = INT
        lib.kmeans_trace_stop.argtypes = []
        lib.kmeans_trace_stop.restype = INT
        lib.kmeans_update_partial.argtypes = [P, P, I64, I64, I64, P, P, P, SZ, U64, P]
        lib.kmeans_update_partial.restype = INT
        lib.kmeans_lloyd_iter_partial.argtypes = [P, P, P, P, P, P, P, I64, I64, I64, P, SZ, U64, P]
        lib.kmeans_lloyd_iter_partial.restype = INT
        lib.kmeans_reduce_partials.argtypes = [P, P, P, INT, I64, I64, P, P, P, P, P]
        lib.kmeans_reduce_partials.restype = INT
        lib.kmeanspp_shard_exchange_bytes.argtypes = [INT, I64]
        lib.kmeanspp_shard_exchange_bytes.restype = SZ
        lib.kmeanspp_shard_first.argtypes = [P, I64, I64, I64, I64, INT, U64, P, P, SZ, P]
        lib.kmeanspp_shard_first.restype = INT
        lib.kmeanspp_shard_pick.argtypes = [P, I64, I64, I64, INT, U64, I64, P, INT, INT, P, P, SZ, P]
        lib.kmeanspp_shard_pick.restype = INT
        lib.kmeanspp_shard_dist.argtypes = [P, I64, I64, INT, INT, P, INT, P, P, SZ, P]
        lib.kmeanspp_shard_dist.restype = INT
        lib.kmeanspp_shard_commit.argtypes = [I64, I64, INT, INT, P, INT, I64, P, P, P, P, SZ, P]
        lib.kmeanspp_shard_commit.restype = INT
        lib.kmeans_route_workspace_bytes.argtypes = [I64, I64, I64]
        lib.kmeans_route_workspace_bytes.restype = SZ
        lib.kmeans_route.argtypes = [P, INT, I64, I64, I64, P, P, P, P, SZ, P]
        lib.kmeans_route.restype = INT
        lib.kmeans_route_gather.argtypes = [P, I64, INT, P, P, I64, I64, I64, I64, P, P]
        lib.kmeans_route_gather.restype = INT
        lib.kmeans_route_combine.argtypes = [P, INT, P, P, I64, P, P, I64, I64, I64, I64, P, P]
        lib.kmeans_route_combine.restype = INT
        lib.kmeans_route_combine_grad.argtypes = [P, I64, P, INT, P, P, P, I64, I64, I64, I64, P, P, P]
        lib.kmeans_route_combine_grad.restype = INT
        lib.kmeans_linear_workspace_bytes.argtypes = [INT, I64, I64, I64, I64]
        lib.kmeans_linear_workspace_bytes.restype = SZ
        lib.kmeans_linear.argtypes = [P, I64, P, P, P, I64, INT, INT, P, I64, I64, I64, I64, P, P, P, SZ, P]
        lib.kmeans_linear.restype = INT
        lib.kmeans_linear_grad.argtypes = [P, I64, P, I64, P, P, INT, INT, P, I64, I64, I64, I64, P, P, P, P, SZ, P]
        lib.kmeans_linear_grad.restype = INT
        F = ctypes.c_float
        lib.kmeans_gate.argtypes = [P, I64, INT, INT, P, I64, I64, I64, I64, I64, INT, F, P, P, P]
        lib.kmeans_gate.restype = INT
        lib.kmeans_gate_grad.argtypes = [P, P, I64, INT, INT, P, I64, I64, I64, INT, F, P, P]
        lib.kmeans_gate_grad.restype = INT
        lib.kmeans_layernorm_workspace_bytes.argtypes = [I64, I64]
        lib.kmeans_layernorm_workspace_bytes.restype = SZ
        lib.kmeans_layernorm.argtypes = [P, I64, INT, P, P, F, I64, I64, P, P, P, P]
        lib.kmeans_layernorm.restype = INT
        lib.kmeans_layernorm_grad.argtypes = [P, I64, P, I64, INT, P, P, P, P, I64, I64, I64, P, P, P, P, SZ, P]
        lib.kmeans_layernorm_grad.restype = INT
        lib.kmeans_cross_entropy_workspace_bytes.argtypes = [INT, I64, I64, I64]
        lib.kmeans_cross_entropy_workspace_bytes.restype = SZ
        lib.kmeans_cross_entropy.argtypes = [P, I64, P, INT, P, INT, F, I64, I64, I64, P, P, P, SZ, P]
        lib.kmeans_cross_entropy.restype = INT
        lib.kmeans_cross_entropy_grad.argtypes = [P, P, I64, P, INT, P, INT, P, F, I64, I64, I64, P, P, P, SZ, P]
        lib.kmeans_cross_entropy_grad.restype = INT
        _lib = lib
        return lib


def kmeans_status_string(status: int) -> str:
    return load().kmeans_status_string(int(status)).decode()


def kmeans_build_info() -> str:
    return load().kmeans_build_info().decode()


def kmeans_workspace_bytes(op: int, n: int, k: int, d: int) -> int:
    return int(load().kmeans_workspace_bytes(op, n, k, d))


def n_trials_for(k: int) -> int:
    """2 + floor(ln k): the default k-means++ trial count."""
    return 2 + int(math.floor(math.log(k)))


# ----------------------------------------------------------------- helpers
_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _stream_handle(stream) -> ctypes.c_void_p:
    torch = _torch()
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _check(t, name, dtype, shape=None, device=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device (the library has no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def workspace(op: int, n: int, k: int, d: int, device=None):
    """A device workspace big enough for ``op`` on these sizes (uint8 tensor)."""
    torch = _torch()
    nbytes = kmeans_workspace_bytes(op, n, k, d)
    if nbytes == 0:
        raise KMeansError(KMEANS_ERR_INVALID_ARG, "kmeans_workspace_bytes")
    return torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")


def _ws(ws, op, n, k, d, device):
    if ws is None:
        return workspace(op, n, k, d, device)
    _check(ws, "ws", _torch().uint8, device=device)
    return ws


def _raise(status, what):
    if status != KMEANS_OK:
        raise KMeansError(status, what)


# ------------------------------------------------------------- entry points
def _assign(fn_name, op, X, C, labels, best_dist, inertia, ws, seed, stream):
    torch = _torch()
    _check(X, "X", torch.float32)
    n, d = X.shape
    _check(C, "C", torch.float32, device=X.device)
    k = C.shape[0]
    if C.dim() != 2 or C.shape[1] != d:
        raise ValueError("C must be (k, d) with the same d as X")
    if labels is None:
        labels = torch.empty(n, dtype=torch.int64, device=X.device)
    if best_dist is None:
        best_dist = torch.empty(n, dtype=torch.float32, device=X.device)
    if inertia is None:
        inertia = torch.empty(1, dtype=torch.float64, device=X.device)
    _check(labels, "labels", torch.int64, (n,), X.device)
    _check(best_dist, "best_dist", torch.float32, (n,), X.device)
    _check(inertia, "inertia", torch.float64, (1,), X.device)
    ws = _ws(ws, op, n, k, d, X.device)
    st = getattr(load(), fn_name)(_ptr(X), _ptr(C), n, k, d, _ptr(labels), _ptr(best_dist), _ptr(inertia),
                                  _ptr(ws), ws.numel(), seed & (2**64 - 1), _stream_handle(stream))
    _raise(st, fn_name)
    return labels, best_dist, inertia


def kmeans_assign(X, C, labels=None, best_dist=None, inertia=None, ws=None, seed=0, stream=None):
    """Nearest centroid on the tensor cores -> ``(labels, best_dist, inertia)``."""
    return _assign("kmeans_assign", OP_ASSIGN, X, C, labels, best_dist, inertia, ws, seed, stream)


def kmeans_assign_ffma(X, C, labels=None, best_dist=None, inertia=None, ws=None, seed=0, stream=None):
    """The same assignment with float32 FMA on the CUDA cores (comparator)."""
    return _assign("kmeans_assign_ffma", OP_ASSIGN_FFMA, X, C, labels, best_dist, inertia, ws, seed, stream)


def kmeans_assign_3xtf32(X, C, labels=None, best_dist=None, inertia=None, ws=None, seed=0, stream=None):
    """The tensor-core assignment with the 3xTF32 split (comparator of bf16x3)."""
    return _assign("kmeans_assign_3xtf32", OP_ASSIGN_3XTF32, X, C, labels, best_dist, inertia, ws, seed, stream)


def kmeans_assign_noalloc(X, C, labels, best_dist, inertia=None, seed=0, stream=None):
    """``kmeans_assign`` for callers that cannot allocate device memory: the
    library's built-in scratch replaces the workspace, and the caller passes
    the outputs.  Problems needing more than NOALLOC_SCRATCH_BYTES of scratch
    raise KMeansError(KMEANS_ERR_SCRATCH_LIMIT)."""
    torch = _torch()
    _check(X, "X", torch.float32)
    n, d = X.shape
    _check(C, "C", torch.float32, device=X.device)
    k = C.shape[0]
    _check(labels, "labels", torch.int64, (n,), X.device)
    _check(best_dist, "best_dist", torch.float32, (n,), X.device)
    if inertia is not None:
        _check(inertia, "inertia", torch.float64, (1,), X.device)
    st = load().kmeans_assign_noalloc(_ptr(X), _ptr(C), n, k, d, _ptr(labels), _ptr(best_dist), _ptr(inertia),
                                      seed & (2**64 - 1), _stream_handle(stream))
    _raise(st, "kmeans_assign_noalloc")
    return labels, best_dist, inertia


def kmeans_update(X, labels, C_old, C_new=None, counts=None, ws=None, seed=0, stream=None):
    """Mean of members, empty clusters keep ``C_old`` -> ``(C_new, counts)``."""
    torch = _torch()
    _check(X, "X", torch.float32)
    n, d = X.shape
    _check(labels, "labels", torch.int64, (n,), X.device)
    _check(C_old, "C_old", torch.float32, device=X.device)
    k = C_old.shape[0]
    if C_new is None:
        C_new = torch.empty_like(C_old)
    if counts is None:
        counts = torch.empty(k, dtype=torch.int32, device=X.device)
    _check(C_new, "C_new", torch.float32, (k, d), X.device)
    _check(counts, "counts", torch.int32, (k,), X.device)
    ws = _ws(ws, OP_UPDATE, n, k, d, X.device)
    st = load().kmeans_update(_ptr(X), _ptr(labels), _ptr(C_old), _ptr(C_new), _ptr(counts), n, k, d,
                              _ptr(ws), ws.numel(), seed & (2**64 - 1), _stream_handle(stream))
    _raise(st, "kmeans_update")
    return C_new, counts


def _lloyd(fn_name, op, X, C_old, C_new, labels, best_dist, inertia, counts, ws, seed, stream):
    torch = _torch()
    _check(X, "X", torch.float32)
    n, d = X.shape
    _check(C_old, "C_old", torch.float32, device=X.device)
    k = C_old.shape[0]
    if C_new is None:
        C_new = torch.empty_like(C_old)
    if labels is None:
        labels = torch.empty(n, dtype=torch.int64, device=X.device)
    if best_dist is None:
        best_dist = torch.empty(n, dtype=torch.float32, device=X.device)
    if inertia is None:
        inertia = torch.empty(1, dtype=torch.float64, device=X.device)
    if counts is None:
        counts = torch.empty(k, dtype=torch.int32, device=X.device)
    _check(C_new, "C_new", torch.float32, (k, d), X.device)
    _check(labels, "labels", torch.int64, (n,), X.device)
    _check(best_dist, "best_dist", torch.float32, (n,), X.device)
    _check(inertia, "inertia", torch.float64, (1,), X.device)
    _check(counts, "counts", torch.int32, (k,), X.device)
    ws = _ws(ws, op, n, k, d, X.device)
    st = getattr(load(), fn_name)(_ptr(X), _ptr(C_old), _ptr(C_new), _ptr(labels), _ptr(best_dist),
                                  _ptr(inertia), _ptr(counts), n, k, d, _ptr(ws), ws.numel(),
                                  seed & (2**64 - 1), _stream_handle(stream))
    _raise(st, fn_name)
    return C_new, labels, best_dist, inertia, counts


def kmeans_lloyd_iter(X, C_old, C_new=None, labels=None, best_dist=None, inertia=None, counts=None, ws=None,
                      seed=0, stream=None):
    """One Lloyd iteration -> ``(C_new, labels, best_dist, inertia, counts)``."""
    return _lloyd("kmeans_lloyd_iter", OP_LLOYD, X, C_old, C_new, labels, best_dist, inertia, counts, ws, seed,
                  stream)


def kmeans_lloyd_iter_fused(X, C_old, C_new=None, labels=None, best_dist=None, inertia=None, counts=None, ws=None,
                            seed=0, stream=None):
    """One Lloyd iteration with the update fused into the assignment (float
    atomics: C_new is not bitwise reproducible) -> as kmeans_lloyd_iter."""
    return _lloyd("kmeans_lloyd_iter_fused", OP_LLOYD_FUSED, X, C_old, C_new, labels, best_dist, inertia, counts,
                  ws, seed, stream)


def kmeanspp_init(X, k: int, seed: int, n_trials: int = 0, centers=None, indices=None, ws=None, stream=None):
    """Greedy D^2 seeding -> ``(indices, centers)``."""
    torch = _torch()
    _check(X, "X", torch.float32)
    n, d = X.shape
    if indices is None:
        indices = torch.empty(k, dtype=torch.int64, device=X.device)
    if centers is None:
        centers = torch.empty((k, d), dtype=torch.float32, device=X.device)
    _check(indices, "indices", torch.int64, (k,), X.device)
    _check(centers, "centers", torch.float32, (k, d), X.device)
    ws = _ws(ws, OP_KMEANSPP, n, k, d, X.device)
    st = load().kmeanspp_init(_ptr(X), n, d, k, int(n_trials), seed & (2**64 - 1), _ptr(centers), _ptr(indices),
                              _ptr(ws), ws.numel(), _stream_handle(stream))
    _raise(st, "kmeanspp_init")
    return indices, centers


def kmeanspp_rows_read(ws, stream=None) -> int:
    """Rows of X the last seeding on ``ws`` read over its distance passes
    (0: it read every row); synchronises the stream."""
    v = ctypes.c_int64(0)
    _raise(load().kmeanspp_rows_read(_ptr(ws), _stream_handle(stream), ctypes.byref(v)), "kmeanspp_rows_read")
    return int(v.value)


def kmeans_device_status(ws, stream=None) -> int:
    """Synchronise the stream; status of the last call that used ``ws``."""
    return int(load().kmeans_device_status(_ptr(ws), _stream_handle(stream)))


def kmeans_relocate_empty(labels, best_dist, k: int, ws=None, stream=None):
    """Move the samples farthest from their centroids into the empty
    clusters (labels rewritten in place) -> ``labels``."""
    torch = _torch()
    _check(labels, "labels", torch.int64)
    n = labels.shape[0]
    _check(best_dist, "best_dist", torch.float32, (n,), labels.device)
    ws = _ws(ws, OP_RELOCATE, n, k, 1, labels.device)
    st = load().kmeans_relocate_empty(_ptr(labels), _ptr(best_dist), n, int(k), _ptr(ws), ws.numel(),
                                      _stream_handle(stream))
    _raise(st, "kmeans_relocate_empty")
    return labels


def kmeans_fit(X, k: int = None, C=None, init: str = "kmeans++", seed: int = 0, max_iter: int = 300,
               tol: float = 1e-4, labels=None, best_dist=None, counts=None, ws=None, stream=None,
               relocate_empty: bool = False):
    """Lloyd iterations until the relative inertia improvement is at most
    ``tol`` (or ``max_iter``) -> ``(C, labels, best_dist, counts,
    inertia_history, n_iter)``.  ``init="kmeans++"`` seeds ``k`` centroids
    with ``seed``; ``init="given"`` starts from ``C`` (updated in place).
    ``relocate_empty`` passes each iteration's labels through
    kmeans_relocate_empty before the update.
    Synchronises the stream once per iteration."""
    import numpy as np
    torch = _torch()
    _check(X, "X", torch.float32)
    n, d = X.shape
    if init == "kmeans++":
        if k is None:
            raise ValueError("init='kmeans++' needs k")
        if C is None:
            C = torch.empty((int(k), d), dtype=torch.float32, device=X.device)
        code = INIT_KMEANSPP
    elif init == "given":
        if C is None:
            raise ValueError("init='given' needs C")
        code = INIT_GIVEN
    else:
        raise ValueError(f"unknown init {init!r}")
    _check(C, "C", torch.float32, device=X.device)
    k = C.shape[0]
    if labels is None:
        labels = torch.empty(n, dtype=torch.int64, device=X.device)
    if best_dist is None:
        best_dist = torch.empty(n, dtype=torch.float32, device=X.device)
    if counts is None:
        counts = torch.empty(k, dtype=torch.int32, device=X.device)
    if ws is None:
        ws = workspace(OP_FIT, n, k, d, X.device)
    hist = np.zeros(int(max_iter), dtype=np.float64)
    n_iter = ctypes.c_int(0)
    if relocate_empty:
        code |= FIT_RELOCATE_EMPTY
    st = load().kmeans_fit(_ptr(X), _ptr(C), _ptr(labels), _ptr(best_dist), _ptr(counts), n, k, d, code,
                           int(seed) & (2**64 - 1), int(max_iter), float(tol), ctypes.byref(n_iter),
                           hist.ctypes.data_as(ctypes.c_void_p), _ptr(ws), ws.numel(), _stream_handle(stream))
    _raise(st, "kmeans_fit")
    return C, labels, best_dist, counts, hist[:n_iter.value].copy(), n_iter.value


def kmeans_trace_start(capacity: int = 1024) -> None:
    """Time each call's dominant kernel with CUDA events (up to ``capacity``
    launches per kernel kind) until kmeans_trace_stop."""
    _raise(load().kmeans_trace_start(int(capacity)), "kmeans_trace_start")


def kmeans_trace_read(kernel: int):
    """``(ms_total, timed_launches, launches)`` of one traced kernel kind
    (KERNEL_ASSIGN_TC, KERNEL_UPDATE_MEAN, KERNEL_KMEANSPP_DIST); waits for
    the recorded events."""
    ms = ctypes.c_double(0.0)
    timed, seen = ctypes.c_int64(0), ctypes.c_int64(0)
    _raise(load().kmeans_trace_read(int(kernel), ctypes.byref(ms), ctypes.byref(timed), ctypes.byref(seen)),
           "kmeans_trace_read")
    return ms.value, timed.value, seen.value


def kmeans_trace_stop() -> None:
    """Turn tracing off and release its events."""
    _raise(load().kmeans_trace_stop(), "kmeans_trace_stop")


def kmeans_lloyd_iter_host(Xh, Ch, Xd, Cd, C_new, labels, best_dist, counts, C_out_h, labels_h, inertia_h,
                           slices: int = 16, ws=None, inertia=None, copy_stream=None, stream=None,
                           overlap_previous: bool = False, readback_on_copy_stream: bool = False):
    """One Lloyd iteration on inputs that live in pinned host memory.

    The library copies the samples to ``Xd`` in ``slices`` row slices on
    ``copy_stream`` and assigns each slice on ``stream`` as soon as it has
    landed; the update follows, and C_new, the labels and the inertia come
    back to ``C_out_h``, ``labels_h`` and ``inertia_h`` (one float64).  The
    device outputs are kmeans_lloyd_iter's: bit for bit with one slice; with
    more, the distances and inertia within the distance tolerance (each
    slice's pass may split other tiles along K).  Returns an event
    recorded after the last copy.  ``overlap_previous``: the copies may
    overlap earlier work on ``stream`` (the caller guarantees that ``Xd`` and
    ``Cd`` are not in use, e.g. by alternating two sets).
    ``readback_on_copy_stream``: the copies back to the host run on
    ``copy_stream`` after the update (the event is recorded there), so that
    ``stream`` can start the next iteration; the caller leaves ``C_new``,
    ``labels`` and ``inertia`` unchanged until the event.
    Xh, Ch, C_out_h, labels_h, inertia_h: pinned host tensors.
    Xd, Cd, C_new, labels, best_dist, counts: device tensors (preallocated).
    """
    torch = _torch()
    n, d = Xh.shape
    k = Ch.shape[0]
    _check(Xd, "Xd", torch.float32, (n, d))
    _check(Cd, "Cd", torch.float32, (k, d), Xd.device)
    _check(C_new, "C_new", torch.float32, (k, d), Xd.device)
    _check(labels, "labels", torch.int64, (n,), Xd.device)
    _check(best_dist, "best_dist", torch.float32, (n,), Xd.device)
    if counts is not None:
        _check(counts, "counts", torch.int32, (k,), Xd.device)
    for t, name, dt, shape in ((Xh, "Xh", torch.float32, (n, d)), (Ch, "Ch", torch.float32, (k, d)),
                               (C_out_h, "C_out_h", torch.float32, (k, d)), (labels_h, "labels_h", torch.int64, (n,)),
                               (inertia_h, "inertia_h", torch.float64, (1,))):
        if t.is_cuda or t.dtype != dt or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous host tensor {dt} {shape}")
    stream = stream or torch.cuda.current_stream()
    copy_stream = copy_stream or torch.cuda.Stream()
    if inertia is None:
        inertia = torch.empty(1, dtype=torch.float64, device=Xd.device)
    if ws is None:
        ws = workspace(OP_LLOYD, n, k, d, Xd.device)
    st = load().kmeans_lloyd_iter_host(Xh.data_ptr(), Ch.data_ptr(), _ptr(Xd), _ptr(Cd), _ptr(C_new), _ptr(labels),
                                       _ptr(best_dist), _ptr(inertia), _ptr(counts), C_out_h.data_ptr(),
                                       labels_h.data_ptr(), inertia_h.data_ptr(), n, k, d, int(slices),
                                       (HOST_OVERLAP_PREVIOUS if overlap_previous else 0) |
                                       (HOST_READBACK_ON_COPY_STREAM if readback_on_copy_stream else 0), _ptr(ws),
                                       ws.numel(), _stream_handle(stream), _stream_handle(copy_stream))
    _raise(st, "kmeans_lloyd_iter_host")
    done = torch.cuda.Event()
    done.record(copy_stream if readback_on_copy_stream else stream)
    return done


# ------------------------------------------------- samples split across GPUs
def kmeans_update_partial(X, labels, k: int, sums=None, counts=None, ws=None, seed=0, stream=None):
    """One shard's cluster sums (zeros for an empty cluster) and counts ->
    ``(sums (k, d), counts (k,))``."""
    torch = _torch()
    _check(X, "X", torch.float32)
    n, d = X.shape
    _check(labels, "labels", torch.int64, (n,), X.device)
    k = int(k)
    if sums is None:
        sums = torch.empty((k, d), dtype=torch.float32, device=X.device)
    if counts is None:
        counts = torch.empty(k, dtype=torch.int32, device=X.device)
    _check(sums, "sums", torch.float32, (k, d), X.device)
    _check(counts, "counts", torch.int32, (k,), X.device)
    ws = _ws(ws, OP_UPDATE_PARTIAL, n, k, d, X.device)
    st = load().kmeans_update_partial(_ptr(X), _ptr(labels), n, k, d, _ptr(sums), _ptr(counts), _ptr(ws), ws.numel(),
                                      seed & (2**64 - 1), _stream_handle(stream))
    _raise(st, "kmeans_update_partial")
    return sums, counts


def kmeans_lloyd_iter_partial(X, C, labels=None, best_dist=None, inertia=None, sums=None, counts=None, ws=None,
                              seed=0, stream=None):
    """One shard's part of a Lloyd iteration -> ``(sums, counts, labels,
    best_dist, inertia)`` (the shard's assignment and its cluster sums)."""
    torch = _torch()
    _check(X, "X", torch.float32)
    n, d = X.shape
    _check(C, "C", torch.float32, device=X.device)
    k = C.shape[0]
    if C.dim() != 2 or C.shape[1] != d:
        raise ValueError("C must be (k, d) with the same d as X")
    labels = torch.empty(n, dtype=torch.int64, device=X.device) if labels is None else labels
    best_dist = torch.empty(n, dtype=torch.float32, device=X.device) if best_dist is None else best_dist
    inertia = torch.empty(1, dtype=torch.float64, device=X.device) if inertia is None else inertia
    sums = torch.empty((k, d), dtype=torch.float32, device=X.device) if sums is None else sums
    counts = torch.empty(k, dtype=torch.int32, device=X.device) if counts is None else counts
    _check(labels, "labels", torch.int64, (n,), X.device)
    _check(best_dist, "best_dist", torch.float32, (n,), X.device)
    _check(inertia, "inertia", torch.float64, (1,), X.device)
    _check(sums, "sums", torch.float32, (k, d), X.device)
    _check(counts, "counts", torch.int32, (k,), X.device)
    ws = _ws(ws, OP_LLOYD_PARTIAL, n, k, d, X.device)
    st = load().kmeans_lloyd_iter_partial(_ptr(X), _ptr(C), _ptr(labels), _ptr(best_dist), _ptr(inertia), _ptr(sums),
                                          _ptr(counts), n, k, d, _ptr(ws), ws.numel(), seed & (2**64 - 1),
                                          _stream_handle(stream))
    _raise(st, "kmeans_lloyd_iter_partial")
    return sums, counts, labels, best_dist, inertia


def kmeans_reduce_partials(parts, part_counts, C_old, C_new=None, counts=None, part_inertia=None, inertia=None,
                           stream=None):
    """Rank-order sum of ``parts`` (world, rows, d) over the summed
    ``part_counts`` (world, rows); C_old's row where no rank has a member ->
    ``(C_new, counts, inertia)``."""
    torch = _torch()
    _check(parts, "parts", torch.float32)
    world, rows, d = parts.shape
    dev = parts.device
    _check(part_counts, "part_counts", torch.int32, (world, rows), dev)
    _check(C_old, "C_old", torch.float32, (rows, d), dev)
    C_new = torch.empty_like(C_old) if C_new is None else C_new
    counts = torch.empty(rows, dtype=torch.int32, device=dev) if counts is None else counts
    _check(C_new, "C_new", torch.float32, (rows, d), dev)
    _check(counts, "counts", torch.int32, (rows,), dev)
    if part_inertia is not None:
        _check(part_inertia, "part_inertia", torch.float64, (world,), dev)
        inertia = torch.empty(1, dtype=torch.float64, device=dev) if inertia is None else inertia
        _check(inertia, "inertia", torch.float64, (1,), dev)
    st = load().kmeans_reduce_partials(_ptr(parts), _ptr(part_counts), _ptr(part_inertia), world, rows, d,
                                       _ptr(C_old), _ptr(C_new), _ptr(counts),
                                       _ptr(inertia if part_inertia is not None else None), _stream_handle(stream))
    _raise(st, "kmeans_reduce_partials")
    return C_new, counts, inertia


def kmeanspp_shard_exchange_bytes(n_trials: int, d: int) -> int:
    return int(load().kmeanspp_shard_exchange_bytes(int(n_trials), int(d)))


def kmeanspp_shard_first(X, row_offset: int, n_global: int, n_trials: int, seed: int, send, ws, stream=None):
    st = load().kmeanspp_shard_first(_ptr(X), X.shape[0], X.shape[1], int(row_offset), int(n_global), int(n_trials),
                                     int(seed) & (2**64 - 1), _ptr(send), _ptr(ws), ws.numel(), _stream_handle(stream))
    _raise(st, "kmeanspp_shard_first")


def kmeanspp_shard_pick(X, row_offset: int, n_trials: int, seed: int, c: int, totals, rank: int, send, ws,
                        stream=None):
    st = load().kmeanspp_shard_pick(_ptr(X), X.shape[0], X.shape[1], int(row_offset), int(n_trials),
                                    int(seed) & (2**64 - 1), int(c), _ptr(totals), totals.numel(), int(rank),
                                    _ptr(send), _ptr(ws), ws.numel(), _stream_handle(stream))
    _raise(st, "kmeanspp_shard_pick")


def kmeanspp_shard_dist(X, n_trials: int, first: bool, recv, world: int, pot, ws, stream=None):
    st = load().kmeanspp_shard_dist(_ptr(X), X.shape[0], X.shape[1], int(n_trials), 1 if first else 0, _ptr(recv),
                                    int(world), _ptr(pot), _ptr(ws), ws.numel(), _stream_handle(stream))
    _raise(st, "kmeanspp_shard_dist")


def kmeanspp_shard_commit(n: int, d: int, n_trials: int, first: bool, pots, world: int, c: int, indices, centers,
                          total, ws, stream=None):
    st = load().kmeanspp_shard_commit(int(n), int(d), int(n_trials), 1 if first else 0, _ptr(pots), int(world), int(c),
                                      _ptr(indices), _ptr(centers), _ptr(total), _ptr(ws), ws.numel(),
                                      _stream_handle(stream))
    _raise(st, "kmeanspp_shard_commit")


# ----------------------------------------- expert routing and expert products
# A routed layer's calls on a few tokens last microseconds on the GPU, so what
# happens before the launch counts: one look at the tensors decides whether all
# is as it should be, and only if not are they looked at again for the reason.
_codes = {}


def _dtype_code(t, name):
    if not _codes:
        torch = _torch()
        _codes.update({torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16})
    code = _codes.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    return code


def _check_on(t, name, dtype, shape, device):
    """_check for a tensor whose device and shape are known."""
    try:
        if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
            return
    except AttributeError:
        pass
    _check(t, name, dtype, shape, device)


def _check_rows(t, name, dtype, shape, device):
    """A matrix whose rows are contiguous, with any pitch -> its pitch."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, it is on {t.device} (the library has no CPU path)")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    rows, cols = shape
    if t.is_contiguous():
        return max(cols, 1)
    pitch = t.stride(0) if rows > 1 else max(cols, 1)
    if (cols > 1 and t.stride(1) != 1) or pitch < cols:
        raise ValueError(f"{name}: the rows must be contiguous and apart from each other")
    return pitch


def _on_gpu(t, name):
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device (the library has no CPU path)")


def _cuda_matrix(t, name):
    _on_gpu(t, name)
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, got shape {tuple(t.shape)}")


def _addr(t):
    return None if t is None else t.data_ptr()


def _current(device):
    """Handle of the device's current stream."""
    return _torch()._C._cuda_getCurrentRawStream(device.index)


def _elsewhere(device):
    """True where another device is current.  The library's launches and their
    limits are the current device's, and a stream's handle does not name one."""
    return _torch()._C._cuda_getDevice() != device.index


def _on_device(device, fn, *args):
    """``fn(*args)`` with ``device`` as the current one."""
    with _torch().cuda.device(device):
        return fn(*args)


def _stream_on(stream, tensor):
    """``stream`` (a torch stream or a handle) as a torch stream of ``tensor``'s
    device."""
    torch = _torch()
    if not isinstance(stream, torch.cuda.Stream):
        return torch.cuda.ExternalStream(int(stream), device=tensor.device)
    if stream.device != tensor.device:
        raise ValueError(f"stream is on {stream.device}, the tensors are on {tensor.device}")
    return stream


def _on_stream(stream, fn, *args):
    """``fn(*args)`` with ``stream`` as the current stream, so that what it
    allocates belongs to that stream (a block that the current stream has given
    back may still be in use there).  The first argument is a tensor."""
    torch = _torch()
    _on_gpu(args[0], "the first argument")
    with torch.cuda.stream(_stream_on(stream, args[0])):
        return fn(*args)


def _workspace_on(ws, device):
    torch = _torch()
    if not (isinstance(ws, torch.Tensor) and ws.dtype is torch.uint8 and ws.device == device and ws.is_contiguous()):
        _check(ws, "ws", torch.uint8, device=device)


def route_workspace(n: int, topk: int, n_experts: int, device=None):
    """A device workspace for ``kmeans_route`` (uint8 tensor)."""
    nbytes = int(load().kmeans_route_workspace_bytes(n, topk, n_experts))
    if nbytes == 0:
        raise KMeansError(KMEANS_ERR_INVALID_ARG, "kmeans_route_workspace_bytes")
    return _torch().empty(nbytes, dtype=_torch().uint8, device=device or "cuda")


def linear_workspace(op: int, m: int, n: int, k: int, n_experts: int = 1, device=None):
    """A device workspace for ``kmeans_linear`` (OP_LINEAR) or
    ``kmeans_linear_grad`` (OP_LINEAR_GRAD) of m rows, n output and k input
    features (uint8 tensor)."""
    nbytes = int(load().kmeans_linear_workspace_bytes(op, m, n, k, n_experts))
    if nbytes == 0:
        raise KMeansError(KMEANS_ERR_INVALID_ARG, "kmeans_linear_workspace_bytes")
    return _torch().empty(nbytes, dtype=_torch().uint8, device=device or "cuda")


def kmeans_route(experts, n_experts: int, offsets=None, order=None, rows=None, ws=None, stream=None):
    """Slots sorted by expert -> ``(offsets (n_experts + 1,), order (n * topk,),
    rows (n, topk))``, all int32.  ``experts`` (n, topk) or (n,): int32 or int64
    ids, negative where the choice was dropped (kmeans_assign's labels route
    each sample to its cluster)."""
    if stream is not None:
        return _on_stream(stream, kmeans_route, experts, n_experts, offsets, order, rows, ws)
    torch = _torch()
    if not isinstance(experts, torch.Tensor):
        raise TypeError("experts must be a torch.Tensor")
    if experts.dtype is not torch.int64 and experts.dtype is not torch.int32:
        raise TypeError(f"experts must be int32 or int64, got {experts.dtype}")
    if experts.dim() not in (1, 2):
        raise ValueError(f"experts must be (n, topk) or (n,), got {tuple(experts.shape)}")
    dev, n_experts = experts.device, int(n_experts)
    n, topk = experts.shape if experts.dim() == 2 else (experts.shape[0], 1)
    if dev.type != "cuda" or not experts.is_contiguous():
        _check(experts, "experts", experts.dtype)
    if _elsewhere(dev):
        return _on_device(dev, kmeans_route, experts, n_experts, offsets, order, rows, ws)
    if n_experts < 1:
        raise ValueError(f"n_experts must be at least 1, got {n_experts}")
    if offsets is None:
        offsets = torch.empty(n_experts + 1, dtype=torch.int32, device=dev)
    else:
        _check_on(offsets, "offsets", torch.int32, (n_experts + 1,), dev)
    if order is None:
        order = torch.empty(n * topk, dtype=torch.int32, device=dev)
    else:
        _check_on(order, "order", torch.int32, (n * topk,), dev)
    if rows is None:
        rows = torch.empty((n, topk), dtype=torch.int32, device=dev)
    else:
        _check_on(rows, "rows", torch.int32, (n, topk), dev)
    if ws is None:
        ws = route_workspace(n, topk, n_experts, dev)
    else:
        _workspace_on(ws, dev)
    st = (_lib or load()).kmeans_route(_addr(experts), experts.element_size(), n, topk, n_experts, _addr(offsets),
                                       _addr(order), _addr(rows), _addr(ws), ws.numel(), _current(dev))
    _raise(st, "kmeans_route")
    return offsets, order, rows


def _plan(rows, offsets, device):
    torch = _torch()
    if not (isinstance(rows, torch.Tensor) and rows.dim() == 2):
        raise ValueError("rows must be (n, topk), as kmeans_route wrote them")
    if not (isinstance(offsets, torch.Tensor) and offsets.dim() == 1 and offsets.numel() >= 2):
        raise ValueError("offsets must be (n_experts + 1,), as kmeans_route wrote them")
    _check_on(rows, "rows", torch.int32, rows.shape, device)
    _check_on(offsets, "offsets", torch.int32, offsets.shape, device)
    n, topk = rows.shape
    return n, topk, offsets.numel() - 1


def kmeans_route_gather(x, rows, offsets, xs=None, stream=None):
    """The tokens in expert order -> ``xs (n * topk, d)``, zeros in the rows of
    dropped choices.  ``rows`` and ``offsets`` are kmeans_route's."""
    if stream is not None:
        return _on_stream(stream, kmeans_route_gather, x, rows, offsets, xs)
    _cuda_matrix(x, "x")
    code = _dtype_code(x, "x")
    dev, dt = x.device, x.dtype
    if _elsewhere(dev):
        return _on_device(dev, kmeans_route_gather, x, rows, offsets, xs)
    n, topk, n_experts = _plan(rows, offsets, dev)
    d = x.shape[1]
    ldx = _check_rows(x, "x", dt, (n, d), dev)
    if xs is None:
        xs = _torch().empty((n * topk, d), dtype=dt, device=dev)
    else:
        _check_on(xs, "xs", dt, (n * topk, d), dev)
    st = (_lib or load()).kmeans_route_gather(_addr(x), ldx, code, _addr(rows), _addr(offsets), n, topk, n_experts, d,
                                              _addr(xs), _current(dev))
    _raise(st, "kmeans_route_gather")
    return xs


def kmeans_route_combine(ys, rows, offsets, weights=None, residual=None, y=None, stream=None):
    """The experts' rows back per token -> ``y (n, d)``: residual + the sum of
    ``weights`` (n, topk) times the choices' rows of ``ys`` (n * topk, d).
    Without weights, also the gradient of kmeans_route_gather."""
    if stream is not None:
        return _on_stream(stream, kmeans_route_combine, ys, rows, offsets, weights, residual, y)
    torch = _torch()
    _cuda_matrix(ys, "ys")
    code = _dtype_code(ys, "ys")
    dev = ys.device
    if _elsewhere(dev):
        return _on_device(dev, kmeans_route_combine, ys, rows, offsets, weights, residual, y)
    n, topk, n_experts = _plan(rows, offsets, dev)
    d = ys.shape[1]
    _check_on(ys, "ys", ys.dtype, (n * topk, d), dev)
    if weights is not None:
        _check_on(weights, "weights", torch.float32, (n, topk), dev)
    ldr = _check_rows(residual, "residual", ys.dtype, (n, d), dev) if residual is not None else 0
    if y is None:
        y = torch.empty((n, d), dtype=ys.dtype, device=dev)
    else:
        _check_on(y, "y", ys.dtype, (n, d), dev)
    st = (_lib or load()).kmeans_route_combine(_addr(ys), code, _addr(weights), _addr(residual), ldr, _addr(rows),
                                               _addr(offsets), n, topk, n_experts, d, _addr(y), _current(dev))
    _raise(st, "kmeans_route_combine")
    return y


def kmeans_route_combine_grad(dy, ys, rows, offsets, weights, dys=None, dweights=None, stream=None):
    """Gradient of kmeans_route_combine -> ``(dys (n * topk, d), dweights
    (n, topk) float32)``; the residual's gradient is ``dy``."""
    if stream is not None:
        return _on_stream(stream, kmeans_route_combine_grad, dy, ys, rows, offsets, weights, dys, dweights)
    torch = _torch()
    _cuda_matrix(ys, "ys")
    code = _dtype_code(ys, "ys")
    dev = ys.device
    if _elsewhere(dev):
        return _on_device(dev, kmeans_route_combine_grad, dy, ys, rows, offsets, weights, dys, dweights)
    n, topk, n_experts = _plan(rows, offsets, dev)
    d = ys.shape[1]
    _check_on(ys, "ys", ys.dtype, (n * topk, d), dev)
    lddy = _check_rows(dy, "dy", ys.dtype, (n, d), dev)
    _check_on(weights, "weights", torch.float32, (n, topk), dev)
    if dys is None:
        dys = torch.empty((n * topk, d), dtype=ys.dtype, device=dev)
    else:
        _check_on(dys, "dys", ys.dtype, (n * topk, d), dev)
    if dweights is None:
        dweights = torch.empty((n, topk), dtype=torch.float32, device=dev)
    else:
        _check_on(dweights, "dweights", torch.float32, (n, topk), dev)
    st = (_lib or load()).kmeans_route_combine_grad(_addr(dy), lddy, _addr(ys), code, _addr(weights), _addr(rows),
                                                    _addr(offsets), n, topk, n_experts, d, _addr(dys), _addr(dweights),
                                                    _current(dev))
    _raise(st, "kmeans_route_combine_grad")
    return dys, dweights


def _linear_args(x, w, offsets, activation):
    """Checked ``(code, m, n, k, n_experts, activation code, weight shape)``."""
    torch = _torch()
    _cuda_matrix(x, "x")
    code = _dtype_code(x, "x")
    if activation not in ACTIVATIONS:
        raise ValueError(f"unknown activation {activation!r} (one of {', '.join(ACTIVATIONS)})")
    if not isinstance(w, torch.Tensor):
        raise TypeError("w must be a torch.Tensor")
    _check_on(w, "w", x.dtype, w.shape, x.device)
    m, k = x.shape
    if offsets is None:
        if w.dim() != 2 and not (w.dim() == 3 and w.shape[0] == 1):
            raise ValueError(f"w must be (n, k) without offsets, got {tuple(w.shape)}")
        n_experts = 1
    else:
        if w.dim() != 3:
            raise ValueError(f"w must be (n_experts, n, k) with offsets, got {tuple(w.shape)}")
        n_experts = w.shape[0]
        _check_on(offsets, "offsets", torch.int32, (n_experts + 1,), x.device)
    if w.shape[-1] != k:
        raise ValueError(f"w has {w.shape[-1]} input features, x has {k}")
    return code, m, w.shape[-2], k, n_experts, ACTIVATIONS[activation]


def kmeans_linear(x, w, bias=None, residual=None, offsets=None, activation="none", save_pre=False, y=None, pre=None,
                  ws=None, stream=None):
    """``act(x w^T + bias) + residual`` -> ``(y (m, n), pre (m, n) or None)``.

    Dense: w (n, k), bias (n,).  Experts: w (n_experts, n, k), bias (n_experts,
    n) and offsets (n_experts + 1,): rows offsets[e] .. offsets[e + 1] - 1 of x
    are expert e's, rows past the last offset give zeros.  ``activation``:
    none, relu, gelu, gelu_tanh or silu.  ``save_pre`` (or a ``pre`` to write
    into) keeps the values before the activation for kmeans_linear_grad.
    float16 or bfloat16."""
    if stream is not None:
        return _on_stream(stream, kmeans_linear, x, w, bias, residual, offsets, activation, save_pre, y, pre, ws)
    torch = _torch()
    code, m, n, k, n_experts, act = _linear_args(x, w, offsets, activation)
    dev, dt = x.device, x.dtype
    if _elsewhere(dev):
        return _on_device(dev, kmeans_linear, x, w, bias, residual, offsets, activation, save_pre, y, pre, ws)
    ldx = _check_rows(x, "x", dt, (m, k), dev)
    if bias is not None:
        _check_on(bias, "bias", dt, tuple(w.shape[:-1]), dev)
    ldr = _check_rows(residual, "residual", dt, (m, n), dev) if residual is not None else 0
    if y is None:
        y = torch.empty((m, n), dtype=dt, device=dev)
    else:
        _check_on(y, "y", dt, (m, n), dev)
    if pre is not None:
        _check_on(pre, "pre", dt, (m, n), dev)
    elif save_pre:
        pre = torch.empty((m, n), dtype=dt, device=dev)
    if ws is None:
        ws = linear_workspace(OP_LINEAR, m, n, k, n_experts, dev)
    else:
        _workspace_on(ws, dev)
    st = (_lib or load()).kmeans_linear(_addr(x), ldx, _addr(w), _addr(bias), _addr(residual), ldr, code, act,
                                        _addr(offsets), m, n, k, n_experts, _addr(y), _addr(pre), _addr(ws), ws.numel(),
                                        _current(dev))
    _raise(st, "kmeans_linear")
    return y, pre


def kmeans_linear_grad(dy, x, w, pre=None, offsets=None, activation="none", need_dx=True, need_dw=True, need_db=True,
                       dx=None, dw=None, db=None, ws=None, stream=None):
    """Gradient of kmeans_linear -> ``(dx, dw, db)`` (None where not needed);
    ``pre`` is what kmeans_linear kept (not needed without an activation).  The
    residual's gradient is ``dy``."""
    if stream is not None:
        return _on_stream(stream, kmeans_linear_grad, dy, x, w, pre, offsets, activation, need_dx, need_dw, need_db,
                          dx, dw, db, ws)
    torch = _torch()
    code, m, n, k, n_experts, act = _linear_args(x, w, offsets, activation)
    dev, dt = x.device, x.dtype
    if _elsewhere(dev):
        return _on_device(dev, kmeans_linear_grad, dy, x, w, pre, offsets, activation, need_dx, need_dw, need_db, dx,
                          dw, db, ws)
    ldx = _check_rows(x, "x", dt, (m, k), dev)
    lddy = _check_rows(dy, "dy", dt, (m, n), dev)
    if act != ACTIVATIONS["none"]:
        if pre is None:
            raise ValueError(f"activation {activation!r} needs pre")
        _check_on(pre, "pre", dt, (m, n), dev)
    if need_dx:
        if dx is None:
            dx = torch.empty((m, k), dtype=dt, device=dev)
        else:
            _check_on(dx, "dx", dt, (m, k), dev)
    if need_dw:
        if dw is None:
            dw = torch.empty_like(w)
        else:
            _check_on(dw, "dw", dt, tuple(w.shape), dev)
    if need_db:
        if db is None:
            db = torch.empty(w.shape[:-1], dtype=dt, device=dev)
        else:
            _check_on(db, "db", dt, tuple(w.shape[:-1]), dev)
    if ws is None:
        ws = linear_workspace(OP_LINEAR_GRAD, m, n, k, n_experts, dev)
    else:
        _check(ws, "ws", torch.uint8, device=dev)
    dx, dw, db = dx if need_dx else None, dw if need_dw else None, db if need_db else None
    st = (_lib or load()).kmeans_linear_grad(_addr(dy), lddy, _addr(x), ldx, _addr(w), _addr(pre), code, act,
                                             _addr(offsets), m, n, k, n_experts, _addr(dx), _addr(dw), _addr(db),
                                             _addr(ws), ws.numel(), _current(dev))
    _raise(st, "kmeans_linear_grad")
    return dx, dw, db


# --------------------------------- around the experts: gate, norm, cross entropy
def _gate_args(logits, scores, topk, scale):
    """Checked ``(code, n, n_experts, score code)``."""
    _cuda_matrix(logits, "logits")
    code = _dtype_code(logits, "logits")
    if scores not in GATE_SCORES:
        raise ValueError(f"unknown scores {scores!r} (one of {', '.join(GATE_SCORES)})")
    n, n_experts = logits.shape
    if n_experts < 1 or not 0 <= topk <= n_experts:
        raise ValueError(f"topk must be in [0, {n_experts}] for {n_experts} experts, got {topk}")
    if not math.isfinite(scale):
        raise ValueError(f"scale must be finite, got {scale}")
    return code, n, n_experts, GATE_SCORES[scores]


def kmeans_gate(logits, topk: int, scores="softmax", bias=None, groups: int = 1, topk_groups: int = None,
                renormalize=True, scale: float = 1.0, ids=None, weights=None, stream=None):
    """Each token's experts from the router's ``logits`` (n, n_experts) ->
    ``(ids (n, topk) int32, weights (n, topk) float32)``, what kmeans_route and
    kmeans_route_combine take.

    The ``topk`` experts with the largest scores (``softmax`` or ``sigmoid`` of
    the logits) plus ``bias`` (n_experts,) float32, in descending order, equal
    ones by index; of ``groups`` groups of neighbouring experts only the
    ``topk_groups`` (all by default) with the largest sums of their two best
    take part.  The weights are the scores times ``scale``, with ``renormalize``
    divided by their sum.  An expert whose logit or bias is -inf is closed; a
    token with fewer open ones gets ids of -1 with weight 0."""
    if stream is not None:
        return _on_stream(stream, kmeans_gate, logits, topk, scores, bias, groups, topk_groups, renormalize, scale, ids,
                          weights)
    torch = _torch()
    topk, groups, scale = int(topk), int(groups), float(scale)
    code, n, n_experts, kind = _gate_args(logits, scores, topk, scale)
    topk_groups = groups if topk_groups is None else int(topk_groups)
    if groups < 1 or n_experts % groups or not 1 <= topk_groups <= groups:
        raise ValueError(f"groups must divide the {n_experts} experts and topk_groups be one of 1 .. groups, got"
                         f" {groups} and {topk_groups}")
    dev = logits.device
    if _elsewhere(dev):
        return _on_device(dev, kmeans_gate, logits, topk, scores, bias, groups, topk_groups, renormalize, scale, ids,
                          weights)
    ldl = _check_rows(logits, "logits", logits.dtype, (n, n_experts), dev)
    if bias is not None:
        _check_on(bias, "bias", torch.float32, (n_experts,), dev)
    if ids is None:
        ids = torch.empty((n, topk), dtype=torch.int32, device=dev)
    else:
        _check_on(ids, "ids", torch.int32, (n, topk), dev)
    if weights is None:
        weights = torch.empty((n, topk), dtype=torch.float32, device=dev)
    else:
        _check_on(weights, "weights", torch.float32, (n, topk), dev)
    st = (_lib or load()).kmeans_gate(_addr(logits), ldl, code, kind, _addr(bias), n, n_experts, topk, groups,
                                      topk_groups, bool(renormalize), scale, _addr(ids), _addr(weights), _current(dev))
    _raise(st, "kmeans_gate")
    return ids, weights


def kmeans_gate_grad(dweights, logits, ids, scores="softmax", renormalize=True, scale: float = 1.0, dlogits=None,
                     stream=None):
    """Gradient of kmeans_gate's weights -> ``dlogits (n, n_experts)``, from
    ``dweights`` (n, topk) float32 and the logits, ids and options of the
    forward call."""
    if stream is not None:
        return _on_stream(stream, kmeans_gate_grad, dweights, logits, ids, scores, renormalize, scale, dlogits)
    torch = _torch()
    scale = float(scale)
    _cuda_matrix(ids, "ids")
    topk = ids.shape[1]
    code, n, n_experts, kind = _gate_args(logits, scores, topk, scale)
    dev, dt = logits.device, logits.dtype
    if _elsewhere(dev):
        return _on_device(dev, kmeans_gate_grad, dweights, logits, ids, scores, renormalize, scale, dlogits)
    ldl = _check_rows(logits, "logits", dt, (n, n_experts), dev)
    _check_on(ids, "ids", torch.int32, (n, topk), dev)
    _check_on(dweights, "dweights", torch.float32, (n, topk), dev)
    if dlogits is None:
        dlogits = torch.empty((n, n_experts), dtype=dt, device=dev)
    else:
        _check_on(dlogits, "dlogits", dt, (n, n_experts), dev)
    st = (_lib or load()).kmeans_gate_grad(_addr(dweights), _addr(logits), ldl, code, kind, _addr(ids), n, n_experts,
                                           topk, bool(renormalize), scale, _addr(dlogits), _current(dev))
    _raise(st, "kmeans_gate_grad")
    return dlogits


def layernorm_workspace(n: int, d: int, device=None):
    """A device workspace for ``kmeans_layernorm_grad`` (uint8 tensor)."""
    nbytes = int(load().kmeans_layernorm_workspace_bytes(n, d))
    if nbytes == 0:
        raise KMeansError(KMEANS_ERR_INVALID_ARG, "kmeans_layernorm_workspace_bytes")
    return _torch().empty(nbytes, dtype=_torch().uint8, device=device or "cuda")


def kmeans_layernorm(x, weight=None, bias=None, eps: float = 1e-5, save_stats=False, y=None, mean=None, rstd=None,
                     stream=None):
    """``(x - mean) * rstd * weight + bias`` per row of x (n, d) -> ``(y (n, d),
    mean (n,) or None, rstd (n,) or None)``, rstd = 1 / sqrt(variance + eps).
    ``weight`` and ``bias`` (d,) of x's type, 1 and 0 by default.
    ``save_stats`` (or a ``mean`` and ``rstd`` to write into) keeps the rows'
    float32 statistics for kmeans_layernorm_grad."""
    if stream is not None:
        return _on_stream(stream, kmeans_layernorm, x, weight, bias, eps, save_stats, y, mean, rstd)
    torch = _torch()
    _cuda_matrix(x, "x")
    code = _dtype_code(x, "x")
    eps = float(eps)
    if not (eps >= 0 and math.isfinite(eps)):
        raise ValueError(f"eps must be at least 0, got {eps}")
    dev, dt = x.device, x.dtype
    if _elsewhere(dev):
        return _on_device(dev, kmeans_layernorm, x, weight, bias, eps, save_stats, y, mean, rstd)
    n, d = x.shape
    ldx = _check_rows(x, "x", dt, (n, d), dev)
    if weight is not None:
        _check_on(weight, "weight", dt, (d,), dev)
    if bias is not None:
        _check_on(bias, "bias", dt, (d,), dev)
    if y is None:
        y = torch.empty((n, d), dtype=dt, device=dev)
    else:
        _check_on(y, "y", dt, (n, d), dev)
    if mean is not None:
        _check_on(mean, "mean", torch.float32, (n,), dev)
    elif save_stats:
        mean = torch.empty(n, dtype=torch.float32, device=dev)
    if rstd is not None:
        _check_on(rstd, "rstd", torch.float32, (n,), dev)
    elif save_stats:
        rstd = torch.empty(n, dtype=torch.float32, device=dev)
    st = (_lib or load()).kmeans_layernorm(_addr(x), ldx, code, _addr(weight), _addr(bias), eps, n, d, _addr(y),
                                           _addr(mean), _addr(rstd), _current(dev))
    _raise(st, "kmeans_layernorm")
    return y, mean, rstd


def kmeans_layernorm_grad(dy, x, mean, rstd, weight=None, residual=None, need_dx=True, need_dweight=True,
                          need_dbias=True, dx=None, dweight=None, dbias=None, ws=None, stream=None):
    """Gradient of kmeans_layernorm -> ``(dx (n, d), dweight (d,), dbias (d,))``
    (None where not needed).  ``mean`` and ``rstd`` are what it kept;
    ``residual`` (n, d), the gradient that reaches x past the norm, is added to
    dx."""
    if stream is not None:
        return _on_stream(stream, kmeans_layernorm_grad, dy, x, mean, rstd, weight, residual, need_dx, need_dweight,
                          need_dbias, dx, dweight, dbias, ws)
    torch = _torch()
    _cuda_matrix(x, "x")
    code = _dtype_code(x, "x")
    dev, dt = x.device, x.dtype
    if _elsewhere(dev):
        return _on_device(dev, kmeans_layernorm_grad, dy, x, mean, rstd, weight, residual, need_dx, need_dweight,
                          need_dbias, dx, dweight, dbias, ws)
    n, d = x.shape
    ldx = _check_rows(x, "x", dt, (n, d), dev)
    lddy = _check_rows(dy, "dy", dt, (n, d), dev)
    ldr = _check_rows(residual, "residual", dt, (n, d), dev) if residual is not None else 0
    _check_on(mean, "mean", torch.float32, (n,), dev)
    _check_on(rstd, "rstd", torch.float32, (n,), dev)
    if weight is not None:
        _check_on(weight, "weight", dt, (d,), dev)
    outs = []
    for name, t, need, shape in (("dx", dx, need_dx, (n, d)), ("dweight", dweight, need_dweight, (d,)),
                                 ("dbias", dbias, need_dbias, (d,))):
        if need and t is None:
            t = torch.empty(shape, dtype=dt, device=dev)
        elif need:
            _check_on(t, name, dt, shape, dev)
        outs.append(t if need else None)
    if ws is None:
        ws = layernorm_workspace(n, d, dev)
    else:
        _workspace_on(ws, dev)
    dx, dweight, dbias = outs
    st = (_lib or load()).kmeans_layernorm_grad(_addr(dy), lddy, _addr(x), ldx, code, _addr(mean), _addr(rstd),
                                                _addr(weight), _addr(residual), ldr, n, d, _addr(dx), _addr(dweight),
                                                _addr(dbias), _addr(ws), ws.numel(), _current(dev))
    _raise(st, "kmeans_layernorm_grad")
    return dx, dweight, dbias


def cross_entropy_workspace(op: int, m: int, n: int, k: int, device=None):
    """A device workspace for ``kmeans_cross_entropy`` (OP_CROSS_ENTROPY) or
    ``kmeans_cross_entropy_grad`` (OP_CROSS_ENTROPY_GRAD, enough for both) of m
    rows, n classes and k features (uint8 tensor).  Fewer rows may need a larger
    one."""
    nbytes = int(load().kmeans_cross_entropy_workspace_bytes(op, m, n, k))
    if nbytes == 0:
        raise KMeansError(KMEANS_ERR_INVALID_ARG, "kmeans_cross_entropy_workspace_bytes")
    return _torch().empty(nbytes, dtype=_torch().uint8, device=device or "cuda")


def _classes_args(x, w, labels, scale):
    """Checked ``(code, m, n, k, ldx)``; all on x's device."""
    torch = _torch()
    code, dev = _dtype_code(x, "x"), x.device
    m, k = x.shape
    ldx = _check_rows(x, "x", x.dtype, (m, k), dev)
    if not (isinstance(w, torch.Tensor) and w.dim() == 2):
        raise ValueError("w must be (n, k), a row for every class")
    _check_on(w, "w", x.dtype, w.shape, dev)
    if w.shape[1] != k:
        raise ValueError(f"w has {w.shape[1]} features, x has {k}")
    if not isinstance(labels, torch.Tensor):
        raise TypeError("labels must be a torch.Tensor")
    if labels.dtype is not torch.int64 and labels.dtype is not torch.int32:
        raise TypeError(f"labels must be int32 or int64, got {labels.dtype}")
    _check_on(labels, "labels", labels.dtype, (m,), dev)
    if not 0 < scale <= 2.0 ** 127:
        raise ValueError(f"scale must be positive and at most 2^127, got {scale}")
    return code, m, w.shape[0], k, ldx


def kmeans_cross_entropy(x, w, labels, scale: float = 1.0, loss=None, lse=None, ws=None, stream=None):
    """Softmax cross entropy of the rows x (m, k) against the classes w (n, k),
    whose m x n logits ``scale * x w^T`` are never stored -> ``(loss (m,),
    lse (m,))`` float32: the logarithm of the sum of a row's exponentials, and
    that minus its label's logit.

    ``labels`` (m,) int32 or int64; a negative one marks a row that does not
    count: loss and lse 0, and whatever it holds reaches nothing else.  One of n
    or more does not count either, and ``kmeans_device_status(ws)`` reports it.  float16 or bfloat16."""
    if stream is not None:
        return _on_stream(stream, kmeans_cross_entropy, x, w, labels, scale, loss, lse, ws)
    torch = _torch()
    _cuda_matrix(x, "x")
    dev, scale = x.device, float(scale)
    if _elsewhere(dev):
        return _on_device(dev, kmeans_cross_entropy, x, w, labels, scale, loss, lse, ws)
    code, m, n, k, ldx = _classes_args(x, w, labels, scale)
    if loss is None:
        loss = torch.empty(m, dtype=torch.float32, device=dev)
    else:
        _check_on(loss, "loss", torch.float32, (m,), dev)
    if lse is None:
        lse = torch.empty(m, dtype=torch.float32, device=dev)
    else:
        _check_on(lse, "lse", torch.float32, (m,), dev)
    if ws is None:
        ws = cross_entropy_workspace(OP_CROSS_ENTROPY, m, n, k, dev)
    else:
        _workspace_on(ws, dev)
    st = (_lib or load()).kmeans_cross_entropy(_addr(x), ldx, _addr(w), code, _addr(labels), labels.element_size(),
                                               scale, m, n, k, _addr(loss), _addr(lse), _addr(ws), ws.numel(),
                                               _current(dev))
    _raise(st, "kmeans_cross_entropy")
    return loss, lse


def kmeans_cross_entropy_grad(dloss, x, w, labels, lse, scale: float = 1.0, need_dx=True, need_dw=True, dx=None,
                              dw=None, ws=None, stream=None):
    """Gradient of kmeans_cross_entropy's losses times ``dloss`` (m,) float32 ->
    ``(dx (m, k), dw (n, k))`` (None where not needed); ``lse`` is what it
    returned for the same x, w and labels.  For the mean over the rows that
    count, dloss is 1 / their number."""
    if stream is not None:
        return _on_stream(stream, kmeans_cross_entropy_grad, dloss, x, w, labels, lse, scale, need_dx, need_dw, dx, dw,
                          ws)
    torch = _torch()
    _cuda_matrix(x, "x")
    dev, dt, scale = x.device, x.dtype, float(scale)
    if _elsewhere(dev):
        return _on_device(dev, kmeans_cross_entropy_grad, dloss, x, w, labels, lse, scale, need_dx, need_dw, dx, dw, ws)
    code, m, n, k, ldx = _classes_args(x, w, labels, scale)
    _check_on(dloss, "dloss", torch.float32, (m,), dev)
    _check_on(lse, "lse", torch.float32, (m,), dev)
    if need_dx:
        if dx is None:
            dx = torch.empty((m, k), dtype=dt, device=dev)
        else:
            _check_on(dx, "dx", dt, (m, k), dev)
    if need_dw:
        if dw is None:
            dw = torch.empty((n, k), dtype=dt, device=dev)
        else:
            _check_on(dw, "dw", dt, (n, k), dev)
    if ws is None:
        ws = cross_entropy_workspace(OP_CROSS_ENTROPY_GRAD, m, n, k, dev)
    else:
        _workspace_on(ws, dev)
    dx, dw = dx if need_dx else None, dw if need_dw else None
    st = (_lib or load()).kmeans_cross_entropy_grad(_addr(dloss), _addr(x), ldx, _addr(w), code, _addr(labels),
                                                    labels.element_size(), _addr(lse), scale, m, n, k, _addr(dx),
                                                    _addr(dw), _addr(ws), ws.numel(), _current(dev))
    _raise(st, "kmeans_cross_entropy_grad")
    return dx, dw
