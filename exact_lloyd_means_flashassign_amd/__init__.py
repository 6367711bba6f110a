"""Python binding of libfk: exact Lloyd k-means on MI355X (gfx950).

A thin ctypes layer over the C ABI in ``include/fk.h``: the functions carry the
same names, check tensor dtypes, devices and shapes, pass raw pointers and the
current torch stream, and raise ``FkError`` on a non-zero status.  Every step
of the computation runs in the HIP kernels of ``libfk.so``; torch is used only
for device memory and streams.  If ``libfk.so`` has not been built, ``load()``
raises -- there is no fallback path.

Each thread caches a workspace per (device, stream) and reuses it in every call
on that stream that does not pass its own ``workspace`` (a thread's calls on
one stream run in order, so they may share it); a call that a graph records has
one of its own.
"""
from __future__ import annotations

import ctypes
import os
import re
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfk.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "fk.h")

METRICS = {"l2": 0, "cosine": 1, "inner_product": 2, "spherical": 3}
SCORES = {"fp32": 0, "split_bf16": 1}
DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
GATES = {"chosen": 0, "all": 1}
PHASES = ("prep", "assign", "recheck", "sort", "reduce", "finalize", "h2d")
MAX_K = 65536
MAX_D = 4096


class FkError(RuntimeError):
    """A non-zero fk_status, with the library's message."""

    def __init__(self, status: int, message: str):
        self.status = status
        super().__init__(f"{_status_name(status)}: {message}")


class _Profile(ctypes.Structure):
    _fields_ = [("calls", ctypes.c_int64 * len(PHASES)), ("ms", ctypes.c_double * len(PHASES)),
                ("rechecked", ctypes.c_int64), ("paired", ctypes.c_int64), ("windowed", ctypes.c_int64),
                ("assigned", ctypes.c_int64)]


class _FitInfo(ctypes.Structure):
    _fields_ = [("k_used", ctypes.c_int32), ("iterations", ctypes.c_int32), ("last_shift", ctypes.c_double)]


class _LinearShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("dtype", "ydtype", "bias_dtype", "act", "groups", "share")] + \
               [(n, ctypes.c_int64) for n in ("M", "N", "K", "ldx", "ldw", "ldr", "ldy", "ldpre")]


_lib = None


def load():
    """Load libfk.so (raises FkError if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise FkError(-1, f"{LIB_PATH} is not built; run __graft_entry__.build() first")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.fk_workspace_size.argtypes = [I64, I32, I32, I32, I64]
    lib.fk_workspace_size.restype = SZ
    lib.fk_assign.argtypes = [P, I64, I32, P, I32, I32, I32, P, P, P, SZ, P]
    lib.fk_sort_inverse.argtypes = [P, I64, I32, P, P, P, SZ, P]
    lib.fk_update.argtypes = [P, I64, I32, P, I32, I32, P, P, P, P, SZ, P]
    lib.fk_lloyd_iter.argtypes = [P, I64, I32, P, I32, I32, I32, P, P, P, P, P, SZ, P]
    lib.fk_lloyd_iter_noalloc.argtypes = [P, I64, I32, P, I32, I32, I32, P, P, P, P, P]
    lib.fk_lloyd_iter_stream.argtypes = [P, I64, I32, P, I32, I32, I32, I64, P, P, P, P, SZ, P]
    lib.fk_fit_workspace_size.argtypes = [I64, I32, I32, I32]
    lib.fk_fit_workspace_size.restype = SZ
    lib.fk_fit.argtypes = [P, I64, I32, I32, I32, I32, P, ctypes.c_uint64, I32, ctypes.c_double, P, P, P,
                           ctypes.POINTER(_FitInfo), P, SZ, P]
    lib.fk_ivf_workspace_size.argtypes = [I64, I32, I32, I32]
    lib.fk_ivf_workspace_size.restype = SZ
    lib.fk_ivf_build.argtypes = [P, I64, I32, I32, I32, I32, I32, P, ctypes.c_uint64, P, P, P, P,
                                 ctypes.POINTER(ctypes.c_int32), P, SZ, P]
    lib.fk_knn_workspace_size.argtypes = [I64, I32, I64, I32, I32]
    lib.fk_knn_workspace_size.restype = SZ
    lib.fk_knn.argtypes = [P, I64, I32, P, I64, I32, I32, I32, P, P, P, SZ, P]
    F32 = ctypes.c_float
    lib.fk_layer_norm.argtypes = [I32, I32, P, I64, I64, I32, P, P, F32, P, I64, P, P, P]
    lib.fk_layer_norm_backward_workspace_size.argtypes = [I64, I32]
    lib.fk_layer_norm_backward_workspace_size.restype = SZ
    lib.fk_layer_norm_backward.argtypes = [I32, I32, P, I64, P, I64, I64, I32, P, P, P, P, I64, P, P, P, SZ, P]
    lib.fk_route_workspace_size.argtypes = [I64, I32]
    lib.fk_route_workspace_size.restype = SZ
    lib.fk_route.argtypes = [I32, P, I64, I64, I32, I32, I32, P, P, P, P, P, P, P, SZ, P]
    lib.fk_route_backward.argtypes = [I32, P, I64, I64, I32, I32, I32, P, P, P, P, P, P, P, P]
    lib.fk_linear_workspace_size.argtypes = [ctypes.POINTER(_LinearShape), I32]
    lib.fk_linear_workspace_size.restype = SZ
    lib.fk_linear.argtypes = [ctypes.POINTER(_LinearShape), P, P, P, P, P, P, P, P, P, SZ, P]
    lib.fk_linear_backward.argtypes = [ctypes.POINTER(_LinearShape), P, P, P, P, P, P, P, P, P, P, SZ, P]
    lib.fk_combine.argtypes = [I32, P, I64, I32, I32, P, P, I64, P, I64, P]
    lib.fk_combine_backward.argtypes = [I32, P, I64, P, I64, I32, I32, P, P, P, P]
    for f in ("fk_layer_norm", "fk_layer_norm_backward", "fk_route", "fk_route_backward", "fk_linear",
              "fk_linear_backward", "fk_combine", "fk_combine_backward"):
        getattr(lib, f).restype = ctypes.c_int
    for f in ("fk_assign", "fk_sort_inverse", "fk_update", "fk_lloyd_iter", "fk_lloyd_iter_noalloc", "fk_lloyd_iter_stream",
              "fk_fit", "fk_ivf_build", "fk_knn", "fk_profile_enable", "fk_profile_read"):
        getattr(lib, f).restype = ctypes.c_int
    lib.fk_status_str.argtypes = [I32]
    lib.fk_status_str.restype = ctypes.c_char_p
    lib.fk_last_error.argtypes = []
    lib.fk_last_error.restype = ctypes.c_char_p
    lib.fk_profile_enable.argtypes = [I32]
    lib.fk_profile_read.argtypes = [ctypes.POINTER(_Profile)]
    _lib = lib
    return lib


def declared_symbols() -> list:
    """Names of the functions include/fk.h declares."""
    with open(HEADER_PATH) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(fk_[a-z_]+)\s*\(", text)))


def _status_name(s: int) -> str:
    if _lib is None:
        return f"status {s}"
    return _lib.fk_status_str(s).decode()


def fk_status_str(status: int) -> str:
    return load().fk_status_str(int(status)).decode()


def _check(status: int):
    if status != 0:
        raise FkError(status, load().fk_last_error().decode())


def _metric(m) -> int:
    if isinstance(m, int):
        return m
    try:
        return METRICS[m]
    except KeyError:
        raise ValueError(f"unknown metric {m!r}") from None


def _score(s) -> int:
    if isinstance(s, int):
        return s
    try:
        return SCORES[s]
    except KeyError:
        raise ValueError(f"unknown score mode {s!r}") from None


def _dev(t, name, dtype, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def _host_pinned(t, name, dtype, shape=None):
    if not isinstance(t, torch.Tensor) or t.is_cuda:
        raise ValueError(f"{name} must be a host tensor")
    if t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype}")
    if not t.is_pinned():
        raise ValueError(f"{name} must be pinned (pin_memory=True)")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


class _Buffers(threading.local):
    """A thread's scratch buffers by (device index, stream).  The calls release
    the interpreter's lock while they enqueue their kernels, so two threads that
    use one stream (the caller's and the autograd engine's, for one) may enqueue
    theirs in turns: each has buffers of its own, which go when it ends."""

    def __init__(self):
        self.by_stream = {}

    def __len__(self):
        return len(self.by_stream)

    def clear(self):
        self.by_stream.clear()


_ws_cache = _Buffers()


def _capturing(d: int, stream: int) -> bool:
    """Whether `stream`, the current one of device index d, is recording a graph
    (the default stream, 0, cannot)."""
    if stream == 0:
        return False
    if torch.cuda.current_device() == d:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.device(d):
        return torch.cuda.is_current_stream_capturing()


def _workspace(nbytes: int, device, workspace=None):
    """(pointer, size, owner) of a 256-byte aligned device workspace of >=
    nbytes; the caller keeps `owner` until its launches are made.  A buffer is
    kept for every stream of a thread and grows with its calls.  A call that a
    graph records gets one of its own instead, from the graph's memory: the
    graph holds its address for as long as it is replayed, whatever the
    stream's own buffer has become by then."""
    if workspace is not None:
        _dev(workspace, "workspace", torch.uint8)
        return workspace.data_ptr(), workspace.numel(), workspace
    dev_index = device.index if device.index is not None else torch.cuda.current_device()
    stream = torch.cuda.current_stream(dev_index).cuda_stream
    if _capturing(dev_index, stream):
        buf = torch.empty(max(nbytes, 1) + 256, dtype=torch.uint8, device=device)
    else:
        key = (dev_index, stream)
        buf = _ws_cache.by_stream.get(key)
        if buf is None or buf.numel() < nbytes + 256:
            _ws_cache.by_stream.pop(key, None)
            buf = torch.empty(max(nbytes, 1) + 256, dtype=torch.uint8, device=device)
            _ws_cache.by_stream[key] = buf
    base = buf.data_ptr()
    pad = (-base) % 256
    return base + pad, buf.numel() - pad, buf


def fk_workspace_size(N: int, d: int, K: int, metric="l2", chunk_rows: int = 0) -> int:
    n = load().fk_workspace_size(int(N), int(d), int(K), _metric(metric), int(chunk_rows))
    if n == 0:
        raise FkError(1, f"sizes outside the limits: N={N} d={d} K={K} chunk_rows={chunk_rows}")
    return int(n)


def _ws_args(N, d, K, metric, device, workspace, chunk_rows=0):
    need = load().fk_workspace_size(int(N), int(d), int(K), _metric(metric), int(chunk_rows))
    if need == 0:
        need = 256  # sizes invalid: the library reports which
    p, n, owner = _workspace(need, device, workspace)
    return ctypes.c_void_p(p), ctypes.c_size_t(n), owner


def fk_assign(X, C, metric="l2", assign=None, min_dist=None, with_min_dist=False, workspace=None, score="fp32"):
    """FlashAssign: returns (assign int32[N], min_dist float32[N] or None).
    score: "fp32" or "split_bf16" (same exact result, different speed)."""
    _dev(X, "X", torch.float32)
    _dev(C, "C", torch.float32)
    if X.dim() != 2 or C.dim() != 2 or X.shape[1] != C.shape[1]:
        raise ValueError("X[N,d] and C[K,d] must be 2-D with the same d")
    N, d = X.shape
    K = C.shape[0]
    if assign is None:
        assign = torch.empty(N, dtype=torch.int32, device=X.device)
    _dev(assign, "assign", torch.int32, (N,))
    if min_dist is None and with_min_dist:
        min_dist = torch.empty(N, dtype=torch.float32, device=X.device)
    if min_dist is not None:
        _dev(min_dist, "min_dist", torch.float32, (N,))
    ws, wsn, _owner = _ws_args(N, d, K, metric, X.device, workspace)
    _check(load().fk_assign(_ptr(X), N, d, _ptr(C), K, _metric(metric), _score(score), _ptr(assign),
                            _ptr(min_dist), ws, wsn, _stream(X.device)))
    return assign, min_dist


def fk_sort_inverse(assign, K: int, perm=None, offsets=None, workspace=None):
    """Inverse index: returns (perm int32[N], offsets int32[K+1])."""
    _dev(assign, "assign", torch.int32)
    N = assign.numel()
    if perm is None:
        perm = torch.empty(N, dtype=torch.int32, device=assign.device)
    if offsets is None:
        offsets = torch.empty(K + 1, dtype=torch.int32, device=assign.device)
    _dev(perm, "perm", torch.int32, (N,))
    _dev(offsets, "offsets", torch.int32, (K + 1,))
    ws, wsn, _owner = _ws_args(N, 1, K, "l2", assign.device, workspace)
    _check(load().fk_sort_inverse(_ptr(assign), N, int(K), _ptr(perm), _ptr(offsets), ws, wsn,
                                  _stream(assign.device)))
    return perm, offsets


def fk_update(X, assign, C_prev, metric="l2", C_out=None, counts=None, workspace=None):
    """Sort-Inverse Update: returns (C_out float32[K,d], counts int32[K])."""
    _dev(X, "X", torch.float32)
    _dev(C_prev, "C_prev", torch.float32)
    N, d = X.shape
    K = C_prev.shape[0]
    _dev(assign, "assign", torch.int32, (N,))
    if C_out is None:
        C_out = torch.empty_like(C_prev)
    if counts is None:
        counts = torch.empty(K, dtype=torch.int32, device=X.device)
    _dev(C_out, "C_out", torch.float32, (K, d))
    _dev(counts, "counts", torch.int32, (K,))
    ws, wsn, _owner = _ws_args(N, d, K, metric, X.device, workspace)
    _check(load().fk_update(_ptr(X), N, d, _ptr(assign), K, _metric(metric), _ptr(C_prev), _ptr(C_out),
                            _ptr(counts), ws, wsn, _stream(X.device)))
    return C_out, counts


def fk_lloyd_iter(X, C_in, metric="l2", assign=None, C_out=None, counts=None, min_dist=None, with_min_dist=False,
                  workspace=None, score="fp32"):
    """One Lloyd iteration: returns (assign, C_out, counts, min_dist or None)."""
    _dev(X, "X", torch.float32)
    _dev(C_in, "C_in", torch.float32)
    if X.dim() != 2 or C_in.dim() != 2 or X.shape[1] != C_in.shape[1]:
        raise ValueError("X[N,d] and C[K,d] must be 2-D with the same d")
    N, d = X.shape
    K = C_in.shape[0]
    if assign is None:
        assign = torch.empty(N, dtype=torch.int32, device=X.device)
    if C_out is None:
        C_out = torch.empty_like(C_in)
    if counts is None:
        counts = torch.empty(K, dtype=torch.int32, device=X.device)
    if min_dist is None and with_min_dist:
        min_dist = torch.empty(N, dtype=torch.float32, device=X.device)
    _dev(assign, "assign", torch.int32, (N,))
    _dev(C_out, "C_out", torch.float32, (K, d))
    _dev(counts, "counts", torch.int32, (K,))
    if min_dist is not None:
        _dev(min_dist, "min_dist", torch.float32, (N,))
    ws, wsn, _owner = _ws_args(N, d, K, metric, X.device, workspace)
    _check(load().fk_lloyd_iter(_ptr(X), N, d, _ptr(C_in), K, _metric(metric), _score(score), _ptr(assign),
                                _ptr(min_dist), _ptr(C_out), _ptr(counts), ws, wsn, _stream(X.device)))
    return assign, C_out, counts, min_dist


NOALLOC_SCRATCH_BYTES = 128 << 20  # FK_NOALLOC_SCRATCH_BYTES of include/fk.h


def fk_lloyd_iter_noalloc(X, C_in, assign, C_out, counts, metric="l2", min_dist=None, score="fp32"):
    """One Lloyd iteration that allocates nothing: the library's static
    per-device scratch replaces the workspace (sizes up to
    NOALLOC_SCRATCH_BYTES of workspace; calls that overlap on one device
    race).  Every output is the caller's.  Returns (assign, C_out, counts,
    min_dist)."""
    _dev(X, "X", torch.float32)
    _dev(C_in, "C_in", torch.float32)
    if X.dim() != 2 or C_in.dim() != 2 or X.shape[1] != C_in.shape[1]:
        raise ValueError("X[N,d] and C[K,d] must be 2-D with the same d")
    N, d = X.shape
    K = C_in.shape[0]
    _dev(assign, "assign", torch.int32, (N,))
    _dev(C_out, "C_out", torch.float32, (K, d))
    _dev(counts, "counts", torch.int32, (K,))
    if min_dist is not None:
        _dev(min_dist, "min_dist", torch.float32, (N,))
    _check(load().fk_lloyd_iter_noalloc(_ptr(X), N, d, _ptr(C_in), K, _metric(metric), _score(score), _ptr(assign),
                                        _ptr(min_dist), _ptr(C_out), _ptr(counts), _stream(X.device)))
    return assign, C_out, counts, min_dist


def fk_lloyd_iter_stream(X_host, C_in, chunk_rows: int, metric="l2", assign_host=None, C_out=None, counts=None,
                         workspace=None, score="fp32"):
    """Out-of-core iteration from pinned host X: returns (C_out, counts).
    assign_host, if given, must be a pinned int32[N] host tensor."""
    _host_pinned(X_host, "X_host", torch.float32)
    _dev(C_in, "C_in", torch.float32)
    N, d = X_host.shape
    K = C_in.shape[0]
    if assign_host is not None:
        _host_pinned(assign_host, "assign_host", torch.int32, (N,))
    if C_out is None:
        C_out = torch.empty_like(C_in)
    if counts is None:
        counts = torch.empty(K, dtype=torch.int32, device=C_in.device)
    _dev(C_out, "C_out", torch.float32, (K, d))
    _dev(counts, "counts", torch.int32, (K,))
    ws, wsn, _owner = _ws_args(N, d, K, metric, C_in.device, workspace, chunk_rows=chunk_rows)
    _check(load().fk_lloyd_iter_stream(_ptr(X_host), N, d, _ptr(C_in), K, _metric(metric), _score(score),
                                       int(chunk_rows), _ptr(assign_host), _ptr(C_out), _ptr(counts), ws, wsn,
                                       _stream(C_in.device)))
    return C_out, counts


def fk_fit_workspace_size(N: int, d: int, K: int, metric="l2") -> int:
    n = load().fk_fit_workspace_size(int(N), int(d), int(K), _metric(metric))
    if n == 0:
        raise FkError(1, f"sizes outside the limits: N={N} d={d} K={K}")
    return int(n)


def fk_fit(X, C_init=None, n_iter: int = 20, metric="l2", K=None, seed: int = 0, tol: float = -1.0, assign=None,
           C_out=None, counts=None, workspace=None, score="fp32", with_info=False):
    """Lloyd k-means: up to n_iter iterations from C_init, or (C_init None)
    from K' = min(K, N) rows of X drawn with `seed`; with tol >= 0 it stops
    once no centroid moves by more than tol (squared L2).  Returns (C_out
    [K', d], assign, counts [K']) and, with with_info, a dict with k_used,
    iterations and last_shift as well."""
    _dev(X, "X", torch.float32)
    if X.dim() != 2:
        raise ValueError("X must be 2-D")
    N, d = X.shape
    if C_init is not None:
        _dev(C_init, "C_init", torch.float32)
        if C_init.dim() != 2 or C_init.shape[1] != d:
            raise ValueError("C_init must be [K, d] with the d of X")
        K = C_init.shape[0]
    elif K is None:
        raise ValueError("give C_init or K")
    K = int(K)
    Ku = K if C_init is not None else min(K, int(N))
    if assign is None:
        assign = torch.empty(N, dtype=torch.int32, device=X.device)
    if C_out is None:
        C_out = torch.empty((max(Ku, 1), d), dtype=torch.float32, device=X.device)
    if counts is None:
        counts = torch.empty(max(Ku, 1), dtype=torch.int32, device=X.device)
    _dev(assign, "assign", torch.int32, (N,))
    _dev(C_out, "C_out", torch.float32)
    _dev(counts, "counts", torch.int32)
    if C_out.numel() < Ku * d or counts.numel() < Ku:
        raise ValueError("C_out and counts must hold K' rows")
    need = load().fk_fit_workspace_size(int(N), int(d), K, _metric(metric)) or 256
    p, n, _owner = _workspace(need, X.device, workspace)
    info = _FitInfo()
    _check(load().fk_fit(_ptr(X), N, d, K, _metric(metric), _score(score), _ptr(C_init), int(seed) & (2 ** 64 - 1),
                         int(n_iter), float(tol), _ptr(C_out), _ptr(assign), _ptr(counts), ctypes.byref(info),
                         ctypes.c_void_p(p), ctypes.c_size_t(n), _stream(X.device)))
    out = (C_out[:info.k_used], assign, counts[:info.k_used])
    if with_info:
        return out + ({"k_used": int(info.k_used), "iterations": int(info.iterations),
                       "last_shift": float(info.last_shift)},)
    return out


def fk_ivf_workspace_size(N: int, d: int, nlist: int, metric="l2") -> int:
    n = load().fk_ivf_workspace_size(int(N), int(d), int(nlist), _metric(metric))
    if n == 0:
        raise FkError(1, f"sizes outside the limits: N={N} d={d} nlist={nlist}")
    return int(n)


def fk_ivf_build(X, nlist: int, init_idx=None, n_iter: int = 20, metric="l2", seed: int = 0, workspace=None,
                 score="fp32"):
    """IVF-Flat build: returns a dict with centroids [nl, d], offsets [nl+1],
    ids [N] and data [N, d] (rows grouped by cell), where nl = min(nlist, N)
    (the library clamps it as the FlashLib guide does); init_idx holds the
    quantizer's initial rows (host ints, at least nl of them), or None for
    nl rows drawn with `seed`."""
    import numpy as np
    _dev(X, "X", torch.float32)
    if X.dim() != 2:
        raise ValueError("X must be 2-D")
    N, d = X.shape
    nlist = int(nlist)
    idx = None
    if init_idx is not None:
        idx = np.ascontiguousarray(np.asarray(init_idx, dtype=np.int32))
        if idx.ndim != 1 or idx.shape[0] < min(nlist, int(N)):
            raise ValueError(f"init_idx has {idx.shape[0]} entries, {min(nlist, int(N))} needed")
    dev = X.device
    rows = max(1, min(nlist, int(N)))
    out = {"centroids": torch.empty((rows, d), dtype=torch.float32, device=dev),
           "offsets": torch.empty(rows + 1, dtype=torch.int32, device=dev),
           "ids": torch.empty(N, dtype=torch.int32, device=dev),
           "data": torch.empty((N, d), dtype=torch.float32, device=dev)}
    need = load().fk_ivf_workspace_size(int(N), int(d), nlist, _metric(metric)) or 256
    p, n, _owner = _workspace(need, dev, workspace)
    nl = ctypes.c_int32(0)
    _check(load().fk_ivf_build(_ptr(X), N, d, nlist, _metric(metric), _score(score), int(n_iter),
                               None if idx is None else ctypes.c_void_p(idx.ctypes.data), int(seed) & (2 ** 64 - 1),
                               _ptr(out["centroids"]), _ptr(out["offsets"]), _ptr(out["ids"]), _ptr(out["data"]),
                               ctypes.byref(nl), ctypes.c_void_p(p), ctypes.c_size_t(n), _stream(dev)))
    out["nlist"] = int(nl.value)
    return out


def fk_knn_workspace_size(M: int, d: int, Ndb: int, k: int, metric="l2") -> int:
    n = load().fk_knn_workspace_size(int(M), int(d), int(Ndb), int(k), _metric(metric))
    if n == 0:
        raise FkError(1, f"sizes outside the limits: M={M} d={d} Ndb={Ndb} k={k}")
    return int(n)


def fk_knn(Q, DB, k: int, metric="l2", idx=None, dist=None, workspace=None, score="fp32"):
    """Exact k nearest database rows of every query: returns (idx [M, k] int32,
    dist [M, k] fp32), nearest first (lower row index first on equal
    distances); with k above the database size the library clamps it as the
    FlashLib backend does and the columns past Ndb hold -1 and +inf."""
    _dev(Q, "Q", torch.float32)
    _dev(DB, "DB", torch.float32)
    if Q.dim() != 2 or DB.dim() != 2 or Q.shape[1] != DB.shape[1]:
        raise ValueError("Q[M,d] and DB[Ndb,d] must be 2-D with the same d")
    M, d = Q.shape
    Ndb = DB.shape[0]
    k = int(k)
    if idx is None:
        idx = torch.empty((M, k), dtype=torch.int32, device=Q.device)
    if dist is None:
        dist = torch.empty((M, k), dtype=torch.float32, device=Q.device)
    _dev(idx, "idx", torch.int32, (M, k))
    _dev(dist, "dist", torch.float32, (M, k))
    need = load().fk_knn_workspace_size(int(M), int(d), int(Ndb), k, _metric(metric)) or 256
    p, n, _owner = _workspace(need, Q.device, workspace)
    _check(load().fk_knn(_ptr(Q), M, d, _ptr(DB), Ndb, k, _metric(metric), _score(score), _ptr(idx), _ptr(dist),
                         ctypes.c_void_p(p), ctypes.c_size_t(n), _stream(Q.device)))
    return idx, dist


# ---- the expert block --------------------------------------------------------
#
# Each operator is a forward and a backward call on plain tensors: what a call
# returns has no autograd history, also where its arguments ask for gradients.
# examples/expert_block.py joins the pairs into autograd functions.


def _named(table, name, what) -> int:
    try:
        return table[name]
    except KeyError:
        raise ValueError(f"unknown {what} {name!r}") from None


def _typed(t, name, dtypes):
    """A GPU tensor of one of `dtypes` (any strides)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {', '.join(map(str, dtypes))}, got {t.dtype}")
    return t


def _rows(t, name, dtypes, shape=None):
    """(row stride) of a matrix with contiguous columns."""
    _typed(t, name, dtypes)
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous columns")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{name} has overlapping rows")
    return t.stride(0) if t.shape[0] > 1 else max(1, t.shape[1])


def _one_device(first, *rest) -> int:
    """Index of the tensors' device, which the call runs on."""
    d = first.get_device()
    for t in rest:
        if t is not None and t.get_device() != d:
            raise ValueError(f"tensors are on different devices: {first.device} and {t.device}")
    return d


def _at(t):
    """The address of a tensor, or None."""
    return None if t is None else t.data_ptr()


# the current stream's handle by device index, without a Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda d: torch.cuda.current_stream(d).cuda_stream)


def _run(fn, d, *args):
    """fn(*args, current stream of device d) with d current; raises on an error."""
    stream = _raw_stream(d)
    if torch.cuda.current_device() == d:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(d):
            status = fn(*args, stream)
    if status != 0:
        _check(status)


def _scratch(nbytes, d, workspace):
    """_workspace for device index d."""
    if workspace is None:
        stream = _raw_stream(d)
        buf = None if _capturing(d, stream) else _ws_cache.by_stream.get((d, stream))
        if buf is not None and buf.numel() >= nbytes + 256:
            base = buf.data_ptr()
            pad = -base % 256
            return base + pad, buf.numel() - pad, buf
    return _workspace(nbytes, torch.device("cuda", d), workspace)


_FLOATS = tuple(DTYPES)


def _param(t, name, dtype, shape):
    """A contiguous parameter of type `dtype` or fp32."""
    _typed(t, name, (dtype, torch.float32))
    if not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be contiguous {tuple(shape)}, got {tuple(t.shape)}")
    return t


def fk_layer_norm(X, weight=None, bias=None, eps: float = 1e-5, Y=None):
    """Layer norm over the rows of X[rows, d] (fp32, bf16 or fp16; rows may be
    strided): returns (Y, mean fp32[rows], rstd fp32[rows]).  weight and bias
    [d] are of X's type or fp32, both of the same."""
    ldx = _rows(X, "X", _FLOATS)
    rows, d = X.shape
    params = [t for t in (weight, bias) if t is not None]
    for t, n in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _param(t, n, X.dtype, (d,))
    if len({t.dtype for t in params}) > 1:
        raise ValueError("weight and bias must be of one type")
    wdt = DTYPES[params[0].dtype if params else X.dtype]
    if Y is None:
        Y, ldy = torch.empty((rows, d), dtype=X.dtype, device=X.device), d
    else:
        ldy = _rows(Y, "Y", (X.dtype,), (rows, d))
    mean = torch.empty(rows, dtype=torch.float32, device=X.device)
    rstd = torch.empty(rows, dtype=torch.float32, device=X.device)
    dev = _one_device(X, weight, bias, Y)
    _run(load().fk_layer_norm, dev, DTYPES[X.dtype], wdt, _at(X), ldx, rows, d, _at(weight), _at(bias), float(eps),
         _at(Y), ldy, _at(mean), _at(rstd))
    return Y, mean, rstd


def fk_layer_norm_backward(dY, X, mean, rstd, weight=None, with_bias: bool = True, dX=None, workspace=None,
                           bias_dtype=None):
    """Gradients of fk_layer_norm: returns (dX, dweight, dbias).  dweight and
    dbias are of the weight's type; dbias is None with with_bias=False.  Without
    a weight dweight is None, and so is dbias unless bias_dtype (the rows' type
    or fp32) says which it should be."""
    ldx = _rows(X, "X", _FLOATS)
    rows, d = X.shape
    ldd = _rows(dY, "dY", (X.dtype,), (rows, d))
    _dev(mean, "mean", torch.float32, (rows,))
    _dev(rstd, "rstd", torch.float32, (rows,))
    if dX is None:
        dX = torch.empty((rows, d), dtype=X.dtype, device=X.device)
    lddx = _rows(dX, "dX", (X.dtype,), (rows, d))
    if bias_dtype not in (None, X.dtype, torch.float32):
        raise ValueError(f"bias_dtype must be {X.dtype} or torch.float32")
    dw, pdt = None, bias_dtype
    if weight is not None:
        _param(weight, "weight", X.dtype, (d,))
        if bias_dtype not in (None, weight.dtype):
            raise ValueError("weight and bias must be of one type")
        dw, pdt = torch.empty_like(weight), weight.dtype
    db = torch.empty(d, dtype=pdt, device=X.device) if with_bias and pdt is not None else None
    dev = _one_device(dY, X, mean, rstd, weight, dX, workspace)
    need = load().fk_layer_norm_backward_workspace_size(rows, d) or 256
    p, n, _owner = _scratch(need, dev, workspace)
    _run(load().fk_layer_norm_backward, dev, DTYPES[X.dtype], DTYPES[pdt or X.dtype],
         _at(dY), ldd, _at(X), ldx, rows, d, _at(mean), _at(rstd), _at(weight), _at(dX), lddx, _at(dw), _at(db), p, n)
    return dX, dw, db


def _valid_mask(valid, T):
    if valid is None:
        return None
    _typed(valid, "valid", (torch.bool, torch.uint8))
    if not valid.is_contiguous() or tuple(valid.shape) != (T,):
        raise ValueError(f"valid must be contiguous ({T},)")
    return valid


def fk_route(logits, k: int, norm="chosen", valid=None, workspace=None):
    """Top-k router over logits[T, E]: returns (ids int32[T, k], gates
    fp32[T, k], counts int32[E], losses fp32[2] = balance and z, live int32[1]).
    norm: "chosen" (gates sum to 1) or "all" (softmax over every expert).
    valid: bool or uint8 [T], rows to leave out where it is 0.  A slot without
    an expert has id E and gate 0."""
    ldl = _rows(logits, "logits", _FLOATS)
    T, E = logits.shape
    k = int(k)
    _valid_mask(valid, T)
    dev = _one_device(logits, valid, workspace)
    ids = torch.empty((T, max(k, 0)), dtype=torch.int32, device=logits.device)
    gates = torch.empty((T, max(k, 0)), dtype=torch.float32, device=logits.device)
    counts = torch.empty(E, dtype=torch.int32, device=logits.device)
    losses = torch.empty(2, dtype=torch.float32, device=logits.device)
    live = torch.empty(1, dtype=torch.int32, device=logits.device)
    need = load().fk_route_workspace_size(T, E) or 256
    p, n, _owner = _scratch(need, dev, workspace)
    _run(load().fk_route, dev, DTYPES[logits.dtype], _at(logits), ldl, T, E, k, _named(GATES, norm, "gate norm"),
         _at(valid), _at(ids), _at(gates), _at(counts), _at(losses), _at(live), p, n)
    return ids, gates, counts, losses, live


def fk_route_backward(logits, ids, counts, live, d_gates=None, d_losses=None, norm="chosen", valid=None):
    """Gradient of fk_route's gates and losses: returns d_logits [T, E]."""
    ldl = _rows(logits, "logits", _FLOATS)
    T, E = logits.shape
    _dev(ids, "ids", torch.int32)
    if ids.dim() != 2 or ids.shape[0] != T:
        raise ValueError(f"ids has shape {tuple(ids.shape)}, expected ({T}, k)")
    k = ids.shape[1]
    _dev(counts, "counts", torch.int32, (E,))
    _dev(live, "live", torch.int32, (1,))
    if d_gates is not None:
        _dev(d_gates, "d_gates", torch.float32, (T, k))
    if d_losses is not None:
        _dev(d_losses, "d_losses", torch.float32, (2,))
    _valid_mask(valid, T)
    dev = _one_device(logits, ids, counts, live, d_gates, d_losses, valid)
    d_logits = torch.empty((T, E), dtype=logits.dtype, device=logits.device)
    _run(load().fk_route_backward, dev, DTYPES[logits.dtype], _at(logits), ldl, T, E, k, _named(GATES, norm,
         "gate norm"), _at(valid), _at(ids), _at(counts), _at(live), _at(d_gates), _at(d_losses), _at(d_logits))
    return d_logits


def _linear_problem(X, W, act, slots, offsets, share):
    """The shape struct of a product, its M and the weights' leading shape."""
    h = _LinearShape()
    h.ldx = _rows(X, "X", _FLOATS)
    _typed(W, "W", (X.dtype,))
    grouped = offsets is not None
    if W.dim() != (3 if grouped else 2):
        raise ValueError("W must be [groups, N, K] with offsets, [N, K] without")
    if grouped and not W.is_contiguous():
        raise ValueError("grouped W must be contiguous")
    N, K = W.shape[-2:]
    if X.shape[1] != K:
        raise ValueError(f"X has {X.shape[1]} columns, W {K}")
    h.ldw = K if grouped else _rows(W, "W", (X.dtype,))
    share = int(share)
    M = X.shape[0] * max(share, 1)
    if grouped:
        _dev(offsets, "offsets", torch.int32)
        if offsets.dim() != 1 or offsets.shape[0] < W.shape[0] + 1:
            raise ValueError(f"offsets must hold groups + 1 = {W.shape[0] + 1} entries")
        if slots is not None:
            _dev(slots, "slots", torch.int32, (M,))
    elif slots is not None:
        raise ValueError("slots need offsets and grouped W")
    h.dtype = h.ydtype = h.bias_dtype = DTYPES[X.dtype]
    h.act = _named(ACTS, act, "activation")
    h.groups = W.shape[0] if grouped else 0
    h.share = share
    h.M, h.N, h.K = M, N, K
    h.ldr = h.ldy = h.ldpre = max(N, 1)
    return h


def fk_linear(X, W, bias=None, act="none", residual=None, slots=None, offsets=None, share: int = 1,
              with_pre: bool = False, out_dtype=None, Y=None, workspace=None):
    """Y = act(X W^T + bias) + residual: returns (Y, pre), pre being the
    pre-activations when with_pre is set (fk_linear_backward takes them), else
    None.  W is [N, K], or with offsets [groups, N, K]: then slot
    s = slots[p] of group g (offsets[g] <= p < offsets[g+1]) is row s of Y and
    takes row s // share of X (X holds M / share rows); offsets may have more
    entries than groups + 1 (fk_sort_inverse of E + 1 clusters), and the slots
    past offsets[groups] give zero rows.  Y is of X's type or, with
    out_dtype=torch.float32, fp32."""
    h = _linear_problem(X, W, act, slots, offsets, share)
    shape = (h.M, h.N)
    if Y is None:
        if out_dtype not in (None, X.dtype, torch.float32):
            raise ValueError(f"out_dtype must be {X.dtype} or torch.float32")
        Y = torch.empty(shape, dtype=out_dtype or X.dtype, device=X.device)
    else:
        h.ldy = _rows(Y, "Y", (X.dtype, torch.float32), shape)
    h.ydtype = DTYPES[Y.dtype]
    if out_dtype is not None and Y.dtype != out_dtype:
        raise ValueError(f"Y is {Y.dtype}, out_dtype {out_dtype}")
    if bias is not None:
        _param(bias, "bias", X.dtype, W.shape[:-1])
        h.bias_dtype = DTYPES[bias.dtype]
    if residual is not None:
        h.ldr = _rows(residual, "residual", (X.dtype,), shape)
    pre = torch.empty(shape, dtype=X.dtype, device=X.device) if with_pre else None
    dev = _one_device(X, W, bias, residual, slots, offsets, Y, workspace)
    need = load().fk_linear_workspace_size(ctypes.byref(h), 2 if slots is None else 0) or 256
    p, n, _owner = _scratch(need, dev, workspace)
    _run(load().fk_linear, dev, ctypes.byref(h), _at(X), _at(W), _at(bias), _at(residual), _at(slots), _at(offsets),
         _at(Y), _at(pre), p, n)
    return Y, pre


def fk_linear_backward(dY, X, W, act="none", pre=None, slots=None, offsets=None, share: int = 1,
                       with_dx: bool = True, with_dw: bool = True, with_bias: bool = True, bias_dtype=None,
                       workspace=None):
    """Gradients of fk_linear: returns (dX, dW, dbias), None for those not
    asked for.  dX has a row for each slot (with share > 1, fk_combine without
    gates adds the rows that share one of X); dW and dbias have the shapes of W
    and the bias.  pre: what fk_linear kept (needed unless act is "none").
    dY act'(pre), an fp32 dY too, is rounded to X's type before the products
    (not for dbias); operands in fp32 keep it whole."""
    h = _linear_problem(X, W, act, slots, offsets, share)
    shape = (h.M, h.N)
    h.ldy = _rows(dY, "dY", (X.dtype, torch.float32), shape)
    h.ydtype = DTYPES[dY.dtype]
    if pre is not None:
        h.ldpre = _rows(pre, "pre", (X.dtype,), shape)
    elif h.act != 0:
        raise ValueError(f"act {act!r} needs pre")
    bias_dtype = bias_dtype or X.dtype
    if bias_dtype not in (X.dtype, torch.float32):
        raise ValueError(f"bias_dtype must be {X.dtype} or torch.float32")
    h.bias_dtype = DTYPES[bias_dtype]
    dev = _one_device(dY, X, W, pre, slots, offsets, workspace)
    dX = torch.empty((h.M, h.K), dtype=X.dtype, device=X.device) if with_dx else None
    dW = torch.empty(W.shape, dtype=X.dtype, device=X.device) if with_dw else None
    db = torch.empty(W.shape[:-1], dtype=bias_dtype, device=X.device) if with_bias else None
    need = load().fk_linear_workspace_size(ctypes.byref(h), 3 if slots is None else 1) or 256
    p, n, _owner = _scratch(need, dev, workspace)
    _run(load().fk_linear_backward, dev, ctypes.byref(h), _at(dY), _at(X), _at(W), _at(pre), _at(slots), _at(offsets),
         _at(dX), _at(dW), _at(db), p, n)
    return dX, dW, db


def _gates_of(gates, rows, k):
    if gates is not None:
        _dev(gates, "gates", torch.float32, (rows, k))
    return gates


def fk_combine(Y, k: int, gates=None, residual=None, out=None):
    """out[t] = residual[t] + sum_j gates[t, j] Y[t k + j] (gates None: all 1):
    returns out [rows, d].  Y [rows k, d] is contiguous."""
    k = int(k)
    _typed(Y, "Y", _FLOATS)
    if Y.dim() != 2 or not Y.is_contiguous():
        raise ValueError("Y must be 2-D and contiguous")
    if k < 1 or Y.shape[0] % k != 0:
        raise ValueError(f"Y has {Y.shape[0]} rows, no multiple of k={k}")
    rows, d = Y.shape[0] // k, Y.shape[1]
    _gates_of(gates, rows, k)
    ldr = _rows(residual, "residual", (Y.dtype,), (rows, d)) if residual is not None else d
    if out is None:
        out, ldo = torch.empty((rows, d), dtype=Y.dtype, device=Y.device), d
    else:
        ldo = _rows(out, "out", (Y.dtype,), (rows, d))
    dev = _one_device(Y, gates, residual, out)
    _run(load().fk_combine, dev, DTYPES[Y.dtype], _at(Y), rows, k, d, _at(gates), _at(residual), ldr, _at(out), ldo)
    return out


def fk_combine_backward(dOut, Y, gates):
    """Gradients of fk_combine: returns (dY [rows k, d], dgates fp32[rows, k]),
    dgates None when gates is (the k is then that of Y's rows)."""
    ldo = _rows(dOut, "dOut", _FLOATS)
    rows, d = dOut.shape
    if gates is None:
        _dev(Y, "Y", dOut.dtype)
        if rows == 0 or Y.dim() != 2 or Y.shape[0] % rows != 0 or Y.shape[1] != d:
            raise ValueError(f"Y has shape {tuple(Y.shape)}, expected (rows k, d) for dOut's {tuple(dOut.shape)}")
        k = Y.shape[0] // rows
    else:
        _dev(gates, "gates", torch.float32)
        if gates.dim() != 2 or gates.shape[0] != rows:
            raise ValueError(f"gates has shape {tuple(gates.shape)}, expected ({rows}, k)")
        k = gates.shape[1]
        _dev(Y, "Y", dOut.dtype, (rows * k, d))
    dev = _one_device(dOut, Y, gates)
    dY = torch.empty((rows * k, d), dtype=dOut.dtype, device=dOut.device)
    dgates = None if gates is None else torch.empty((rows, k), dtype=torch.float32, device=dOut.device)
    _run(load().fk_combine_backward, dev, DTYPES[dOut.dtype], _at(dOut), ldo, _at(Y), rows, k, d, _at(gates), _at(dY),
         _at(dgates))
    return dY, dgates


def fk_profile_enable(on: bool = True):
    _check(load().fk_profile_enable(1 if on else 0))


def fk_profile_read() -> dict:
    """Waits for the pending phase events; returns per-phase calls and
    milliseconds, the near-tie points settled by an fp64 compare of two
    centroids ("paired"), of the centroids within their error window
    ("windowed"), or against all K ("rechecked"), and the points assigned."""
    p = _Profile()
    _check(load().fk_profile_read(ctypes.byref(p)))
    return {"calls": {ph: int(p.calls[i]) for i, ph in enumerate(PHASES)},
            "ms": {ph: float(p.ms[i]) for i, ph in enumerate(PHASES)},
            "rechecked": int(p.rechecked), "paired": int(p.paired), "windowed": int(p.windowed),
            "assigned": int(p.assigned)}
