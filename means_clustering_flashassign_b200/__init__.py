"""Exact Lloyd K-Means on B200 (sm_100a): FlashAssign + Sort-Inverse Update.

Thin Python binding of ``libkm.so`` (C ABI in ``include/km.h``).  This module
only marshals arguments: it checks shapes, allocates outputs and workspace with
torch (device memory and streams are the only things torch provides) and calls
the C entry points, which run every step of the computation in CUDA kernels.
There is no CPU or PyTorch fallback: if the library is missing or the GPU is
not an sm_100 part, calls raise.

Method: "Flash-KMeans: Fast and Memory-Efficient Exact K-Means", §2.1
FlashAssign (fused distance tiles + online argmin, no N x K matrix in device
memory), §2.2 Sort-Inverse Update (argsort of the assignment vector +
segmented on-chip reduction), §2.3 Chunked Stream Overlap (host-resident points
streamed in chunks).
"""

from __future__ import annotations

import ctypes
import functools
import os
import threading
from typing import NamedTuple, Optional

import torch

from . import build as _build

__all__ = ["KMError", "library", "library_path", "workspace_size", "assign", "update", "fit", "fit_host",
           "workspace_status", "selftest_timeout", "argsort", "fit_profile", "launch_count", "assign_static",
           "ablation_assign_materialized", "ablation_update_atomic", "plan", "update_accumulate",
           "finalize_sums", "fit_data_parallel", "pack_layout", "exchange_packed", "fit_source", "FitGraph",
           "Quantized", "quantize", "dequantize", "scores", "scores_grad", "Balance", "balance", "balance_grad",
           "soft_workspace_size", "SOFT_SCORES", "SOFT_SCORES_GRAD", "SOFT_BALANCE",
           "OP_ASSIGN", "OP_UPDATE", "OP_FIT", "OP_FIT_HOST",
           "OP_ARGSORT",
           "F32", "BF16", "EXPORTS"]

OP_ASSIGN, OP_UPDATE, OP_FIT, OP_FIT_HOST, OP_ARGSORT = 0, 1, 2, 3, 4
SOFT_SCORES, SOFT_SCORES_GRAD, SOFT_BALANCE = 0, 1, 2
F32, BF16 = 0, 1
STATUS = {0: "KM_OK", 1: "KM_ERR_INVALID_ARG", 2: "KM_ERR_UNSUPPORTED", 3: "KM_ERR_CUDA",
          4: "KM_ERR_WORKSPACE", 5: "KM_ERR_TIMEOUT", 6: "KM_ERR_INJECTED"}
EXPORTS = ["km_version", "km_status_string", "km_last_error", "km_workspace_size", "km_workspace_status",
           "km_assign", "km_update", "km_argsort", "km_fit", "km_fit_profile", "km_fit_timed", "km_fit_host", "km_selftest_timeout",
           "km_launch_count", "km_assign_static", "km_ablation_workspace_size", "km_ablation_assign_materialized",
           "km_ablation_update_atomic", "km_plan_describe", "km_update_accumulate", "km_finalize_sums",
           "km_fit_source", "km_fit_graph_create", "km_fit_graph_launch", "km_fit_graph_elapsed",
           "km_fit_graph_destroy", "km_soft_workspace_size", "km_quantize", "km_dequantize", "km_scores",
           "km_scores_grad", "km_balance", "km_balance_grad"]

_lock = threading.Lock()
_lib = None

# km_chunk_source: const void* (*)(void* user, int64_t row0, int64_t rows, int slot)
CHUNK_SOURCE = ctypes.CFUNCTYPE(ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int)


class KMError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status
        self.message = message


def library_path() -> str:
    return _build.LIB


def library() -> ctypes.CDLL:
    """Load libkm.so (building it first if the sources are newer)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = _build.LIB
            if not _build.up_to_date():
                path = _build.build()
            if not os.path.exists(path):
                raise RuntimeError(f"libkm.so not found at {path}; run means_clustering_flashassign_b200.build")
            L = ctypes.CDLL(path)
            P, I, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
            L.km_version.restype = I
            L.km_status_string.argtypes = [I]
            L.km_status_string.restype = ctypes.c_char_p
            L.km_last_error.restype = ctypes.c_char_p
            L.km_workspace_size.argtypes = [I, I, I64, I, I, I, I64]
            L.km_workspace_size.restype = SZ
            L.km_workspace_status.argtypes = [P, P]
            L.km_assign.argtypes = [P, P, I, I64, I, I, I, P, P, P, P, SZ, P]
            L.km_update.argtypes = [P, P, I, I64, I, I, I, P, P, P, SZ, P]
            L.km_fit.argtypes = [P, P, I, I64, I, I, I, I, P, P, P, P, P, SZ, P]
            L.km_fit_host.argtypes = [P, P, I64, I, I, I, I, I64, P, P, P, P, P, SZ, P]
            L.km_selftest_timeout.argtypes = [P, SZ, I64, P]
            L.km_argsort.argtypes = [P, I64, I, P, P, P, SZ, P]
            L.km_plan_describe.argtypes = [I, I, I64, I, I, I, I64, P]
            L.km_update_accumulate.argtypes = [P, P, I64, I, I, I, P, P, I, P, SZ, P]
            L.km_finalize_sums.argtypes = [P, P, I, I, I, P, P, P, P]
            L.km_ablation_workspace_size.argtypes = [I, I64, I, I, I, I64]
            L.km_ablation_workspace_size.restype = SZ
            L.km_ablation_assign_materialized.argtypes = [P, P, I64, I, I, I, I64, P, P, P, SZ, P]
            L.km_ablation_update_atomic.argtypes = [P, P, I64, I, I, I, P, P, P, SZ, P]
            L.km_fit_profile.argtypes = [P, P, I, I64, I, I, I, I, P, P, P, P, P, SZ, P, P]
            L.km_fit_timed.argtypes = [P, P, I, I64, I, I, I, I, P, P, P, P, P, SZ, P, P]
            L.km_launch_count.restype = ctypes.c_uint64
            L.km_assign_static.argtypes = [P, P, I, I64, I, I, I, P, P, P, P]
            L.km_fit_source.argtypes = [CHUNK_SOURCE, P, P, I64, I, I, I, I, I64, P, P, P, P, P, SZ, P]
            L.km_fit_graph_create.argtypes = [P, P, P, I, I64, I, I, I, I, P, P, P, P, P, SZ, I]
            L.km_fit_graph_launch.argtypes = [P, P]
            L.km_fit_graph_elapsed.argtypes = [P, P]
            L.km_fit_graph_destroy.argtypes = [P]
            L.km_soft_workspace_size.argtypes = [I, I, I64, I, I, I]
            L.km_soft_workspace_size.restype = SZ
            F = ctypes.c_float
            L.km_quantize.argtypes = [P, I, I64, I, I, P, P, P]
            L.km_dequantize.argtypes = [P, P, I, I64, I, I, P, P]
            L.km_scores.argtypes = [P, P, P, P, P, F, I, I64, I, I, I, P, P, SZ, P]
            L.km_scores_grad.argtypes = [P, P, P, P, P, F, I, I64, I, I, I, I, P, P, P, P, SZ, P]
            L.km_balance.argtypes = [P, P, P, I, I64, I, I, I, P, P, P, P, P, P, SZ, P]
            L.km_balance_grad.argtypes = [P, P, P, P, P, P, P, I, I64, I, I, I, P, P]
            for f in EXPORTS:
                getattr(L, f).restype = getattr(L, f).restype or I
            _lib = L
    return _lib


def _check(status: int) -> None:
    if status != 0:
        msg = library().km_last_error().decode(errors="replace")
        raise KMError(status, msg)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"points must be bfloat16 or float32, got {t.dtype}")


def _shape3(X: torch.Tensor, name: str):
    if X.dim() == 2:
        return 1, X.shape[0], X.shape[1], False
    if X.dim() == 3:
        return X.shape[0], X.shape[1], X.shape[2], True
    raise ValueError(f"{name} must be (N, D) or (B, N, D)")


def workspace_size(op: int, B: int, N: int, D: int, K: int, dtype: int, chunk_rows: int = 0) -> int:
    n = library().km_workspace_size(op, B, N, D, K, dtype, chunk_rows)
    if n == 0:
        raise KMError(2, library().km_last_error().decode(errors="replace"))
    return int(n)


def _workspace(op, B, N, D, K, dtype, device, workspace=None, chunk_rows=0):
    need = workspace_size(op, B, N, D, K, dtype, chunk_rows)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    if workspace.numel() < need:
        raise ValueError(f"workspace has {workspace.numel()} bytes, needs {need}")
    return workspace


def _contig_cuda(t: torch.Tensor, name: str) -> torch.Tensor:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _check_tensor(t: torch.Tensor, name: str, device: torch.device, dtype=None, shape=None) -> torch.Tensor:
    """Reject a tensor the kernels would read or write out of place: on
    another device than the points, of another dtype or shape than the call
    writes, or not contiguous (the kernels index it as a dense array)."""
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the points are on {device}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _check_stream(stream, device: torch.device) -> None:
    if stream is not None and stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the points are on {device}")


def assign(X: torch.Tensor, C: torch.Tensor, *, idx=None, mindist=None, want_mindist: bool = True,
           want_objective: bool = True, workspace=None, stream=None):
    """FlashAssign: nearest centroid of every point (lowest index on ties).

    X: (N, D) or (B, N, D) bf16/f32 CUDA tensor; C: (K, D) or (B, K, D), same dtype.
    Returns (idx int32, mindist float32 or None, objective float64 [B] or None).
    """
    B, N, D, K, dt, shp = _assign_args(X, C, idx, mindist, stream)
    with torch.cuda.device(X.device):
        idx = torch.empty(shp, dtype=torch.int32, device=X.device) if idx is None else idx
        if mindist is None and want_mindist:
            mindist = torch.empty(shp, dtype=torch.float32, device=X.device)
        obj = torch.empty(B, dtype=torch.float64, device=X.device) if want_objective else None
        ws = _workspace(OP_ASSIGN, B, N, D, K, dt, X.device, workspace)
        _check_tensor(ws, "workspace", X.device, torch.uint8)
        _check(library().km_assign(_ptr(X), _ptr(C), B, N, D, K, dt, _ptr(idx), _ptr(mindist), _ptr(obj),
                                   _ptr(ws), ws.numel(), _stream(stream)))
    return idx, mindist, obj


def _assign_args(X, C, idx, mindist, stream):
    """Shapes of an assignment call, with every tensor checked against X."""
    _contig_cuda(X, "X"), _contig_cuda(C, "C")
    B, N, D, batched = _shape3(X, "X")
    Bc, K, Dc, _ = _shape3(C, "C")
    if Bc != B or Dc != D or C.dtype != X.dtype:
        raise ValueError("C must match X in batch, D and dtype")
    dt = _dtype_code(X)
    shp = (B, N) if batched else (N,)
    _check_tensor(C, "C", X.device)
    if idx is not None:
        _check_tensor(idx, "idx", X.device, torch.int32, shp)
    if mindist is not None:
        _check_tensor(mindist, "mindist", X.device, torch.float32, shp)
    _check_stream(stream, X.device)
    return B, N, D, K, dt, shp


def assign_static(X: torch.Tensor, C: torch.Tensor, *, idx=None, mindist=None, want_mindist: bool = True,
                  want_objective: bool = True, stream=None):
    """assign() without a workspace: scratch comes from the library's fixed
    16 MiB static device area (for callers that cannot allocate; shapes that
    need more are refused).  Same results as assign()."""
    B, N, D, K, dt, shp = _assign_args(X, C, idx, mindist, stream)
    with torch.cuda.device(X.device):
        idx = torch.empty(shp, dtype=torch.int32, device=X.device) if idx is None else idx
        if mindist is None and want_mindist:
            mindist = torch.empty(shp, dtype=torch.float32, device=X.device)
        obj = torch.empty(B, dtype=torch.float64, device=X.device) if want_objective else None
        _check(library().km_assign_static(_ptr(X), _ptr(C), B, N, D, K, dt, _ptr(idx), _ptr(mindist), _ptr(obj),
                                          _stream(stream)))
    return idx, mindist, obj


def update(X: torch.Tensor, idx: torch.Tensor, C: torch.Tensor, *, counts=None, want_counts: bool = True,
           workspace=None, stream=None):
    """Sort-Inverse Update: C (float32, in: previous, out: new) <- member means.

    Returns (C, counts int32 or None).  C is updated in place.
    """
    _contig_cuda(X, "X"), _contig_cuda(idx, "idx"), _contig_cuda(C, "C")
    B, N, D, batched = _shape3(X, "X")
    Bc, K, Dc, _ = _shape3(C, "C")
    if Bc != B or Dc != D or C.dtype != torch.float32 or idx.dtype != torch.int32:
        raise ValueError("C must be float32 (B, K, D) matching X; idx int32")
    dt = _dtype_code(X)
    _check_tensor(idx, "idx", X.device, torch.int32, (B, N) if batched else (N,))
    _check_tensor(C, "C", X.device)
    kshape = (B, K) if batched else (K,)
    if counts is not None:
        _check_tensor(counts, "counts", X.device, torch.int32, kshape)
    _check_stream(stream, X.device)
    with torch.cuda.device(X.device):
        if counts is None and want_counts:
            counts = torch.empty(kshape, dtype=torch.int32, device=X.device)
        ws = _workspace(OP_UPDATE, B, N, D, K, dt, X.device, workspace)
        _check_tensor(ws, "workspace", X.device, torch.uint8)
        _check(library().km_update(_ptr(X), _ptr(idx), B, N, D, K, dt, _ptr(C), _ptr(counts), _ptr(ws),
                                   ws.numel(), _stream(stream)))
    return C, counts


def argsort(idx: torch.Tensor, K: int, *, workspace=None, stream=None):
    """Stable argsort of an assignment vector by cluster id on the device.

    Returns (perm int32 [N], start int32 [K+1]).
    """
    _contig_cuda(idx, "idx")
    if idx.dtype != torch.int32 or idx.dim() != 1:
        raise ValueError("idx must be a 1-D int32 tensor")
    N = idx.shape[0]
    _check_stream(stream, idx.device)
    with torch.cuda.device(idx.device):
        perm = torch.empty(N, dtype=torch.int32, device=idx.device)
        start = torch.empty(K + 1, dtype=torch.int32, device=idx.device)
        ws = _workspace(OP_ARGSORT, 1, N, 0, K, 0, idx.device, workspace)
        _check_tensor(ws, "workspace", idx.device, torch.uint8)
        _check(library().km_argsort(_ptr(idx), N, K, _ptr(perm), _ptr(start), _ptr(ws), ws.numel(),
                                    _stream(stream)))
    return perm, start


def update_accumulate(X: torch.Tensor, idx: torch.Tensor, sums: torch.Tensor, counts: torch.Tensor, *,
                      zero_first: bool = True, workspace=None, stream=None) -> None:
    """Sort-Inverse Update of one shard added into float64 sums [K, D] and
    float64 counts [K] (zeroed first by default).  sums and counts may be
    views into one buffer (see pack_layout)."""
    _contig_cuda(X, "X"), _contig_cuda(idx, "idx"), _contig_cuda(sums, "sums"), _contig_cuda(counts, "counts")
    if X.dim() != 2 or sums.dim() != 2:
        raise ValueError("X must be [N, D] and sums [K, D]")
    N, D = X.shape
    K = sums.shape[0]
    _check_tensor(idx, "idx", X.device, torch.int32, (N,))
    _check_tensor(sums, "sums", X.device, torch.float64, (K, D))
    _check_tensor(counts, "counts", X.device, torch.float64, (K,))
    _check_stream(stream, X.device)
    dt = _dtype_code(X)
    with torch.cuda.device(X.device):
        ws = _workspace(OP_UPDATE, 1, N, D, K, dt, X.device, workspace)
        _check_tensor(ws, "workspace", X.device, torch.uint8)
        _check(library().km_update_accumulate(_ptr(X), _ptr(idx), N, D, K, dt, _ptr(sums), _ptr(counts),
                                              1 if zero_first else 0, _ptr(ws), ws.numel(), _stream(stream)))


def finalize_sums(sums: torch.Tensor, counts: torch.Tensor, C: torch.Tensor, C_lp: Optional[torch.Tensor] = None,
                  counts_out: Optional[torch.Tensor] = None, *, stream=None) -> None:
    """C = sums / counts where counts > 0 (else kept), in place; C_lp gets the
    dtype copy for the next assign; counts_out the int32 counts.  sums
    float64 [K, D], counts float64 [K], C float32 [K, D]."""
    _contig_cuda(C, "C")
    if C.dim() != 2:
        raise ValueError("C must be [K, D]")
    K, D = C.shape
    dev = C.device
    _check_tensor(C, "C", dev, torch.float32)
    _check_tensor(sums, "sums", dev, torch.float64, (K, D))
    _check_tensor(counts, "counts", dev, torch.float64, (K,))
    if C_lp is not None:
        _check_tensor(C_lp, "C_lp", dev, shape=(K, D))
    if counts_out is not None:
        _check_tensor(counts_out, "counts_out", dev, torch.int32, (K,))
    _check_stream(stream, dev)
    dt = _dtype_code(C_lp) if C_lp is not None else F32
    with torch.cuda.device(dev):
        _check(library().km_finalize_sums(_ptr(sums), _ptr(counts), K, D, dt, _ptr(C), _ptr(C_lp),
                                          _ptr(counts_out), _stream(stream)))


def pack_layout(K: int, D: int) -> dict:
    """Layout of the one float64 buffer a data-parallel iteration exchanges:
    the per-cluster sums [K*D], the counts [K] (exact integers in float64)
    and the objective [1], in that order, so that one all-reduce (sum) adds
    all three across the ranks.  Returns slices into a flat buffer."""
    kd = K * D
    return {"sums": slice(0, kd), "counts": slice(kd, kd + K), "objective": slice(kd + K, kd + K + 1),
            "size": kd + K + 1}


def exchange_packed(buf: torch.Tensor, *, group=None) -> None:
    """Add a packed buffer (pack_layout) across the ranks of `group` in
    place: one all-reduce.  NCCL reduces device tensors directly; a gloo
    group goes through a host copy."""
    import torch.distributed as dist
    if buf.dtype != torch.float64 or buf.dim() != 1 or not buf.is_contiguous():
        raise ValueError("the exchange buffer must be a contiguous 1-D float64 tensor")
    if buf.is_cuda and dist.get_backend(group) == "gloo":
        h = buf.cpu()
        dist.all_reduce(h, group=group)
        buf.copy_(h)
    else:
        dist.all_reduce(buf, group=group)


def fit_data_parallel(X: torch.Tensor, C0: torch.Tensor, iters: int, *, group=None, sync_objective: bool = True):
    """Lloyd iterations over a point set sharded by rows across the ranks of a
    torch.distributed process group: every rank passes its own rows X and the
    same C0.  Per iteration each rank assigns its rows and sums them per
    cluster (float64, deterministic) into one packed buffer (sums, counts,
    objective); one all-reduce adds the ranks' buffers; every rank finalises
    the same sums, so C is the same on all ranks.  The objective history stays
    on the device until the end (no host synchronisation per iteration).
    Returns dict(C float32 [K, D], idx (this rank's rows), counts int32 [K],
    objective float64 [iters]: the whole point set's J_t, on the host when
    sync_objective, else on the device)."""
    _contig_cuda(X, "X"), _contig_cuda(C0, "C0")
    if X.dim() != 2 or C0.dim() != 2 or C0.shape[1] != X.shape[1] or C0.dtype != X.dtype:
        raise ValueError("X [N, D] and C0 [K, D] of one dtype")
    _check_tensor(C0, "C0", X.device)
    N, D = X.shape
    K = C0.shape[0]
    dev = X.device
    lay = pack_layout(K, D)
    with torch.cuda.device(dev):
        C = C0.float().contiguous().clone()
        C_lp = C0.clone()
        buf = torch.empty(lay["size"], dtype=torch.float64, device=dev)
        sums = buf[lay["sums"]].view(K, D)
        cnt = buf[lay["counts"]]
        obj = buf[lay["objective"]]
        counts = torch.empty(K, dtype=torch.int32, device=dev)
        idx = torch.empty(N, dtype=torch.int32, device=dev)
        dt = _dtype_code(X)
        ws_a = _workspace(OP_ASSIGN, 1, N, D, K, dt, dev)
        ws_u = _workspace(OP_UPDATE, 1, N, D, K, dt, dev)
        J = torch.empty(iters, dtype=torch.float64, device=dev)
        L = library()
        s = _stream(None)
        for t in range(iters):
            _check(L.km_assign(_ptr(X), _ptr(C_lp), 1, N, D, K, dt, _ptr(idx), None, _ptr(obj), _ptr(ws_a),
                               ws_a.numel(), s))
            _check(L.km_update_accumulate(_ptr(X), _ptr(idx), N, D, K, dt, _ptr(sums), _ptr(cnt), 1, _ptr(ws_u),
                                          ws_u.numel(), s))
            exchange_packed(buf, group=group)
            _check(L.km_finalize_sums(_ptr(sums), _ptr(cnt), K, D, dt, _ptr(C), _ptr(C_lp), _ptr(counts), s))
            J[t:t + 1].copy_(obj)
    return dict(C=C, idx=idx, counts=counts, objective=J.cpu() if sync_objective else J)


def plan(op: int, B: int, N: int, D: int, K: int, dtype: int, chunk_rows: int = 0) -> dict:
    """The tiling the library would use for this shape (host-only query)."""
    out = (ctypes.c_int64 * 9)()
    _check(library().km_plan_describe(op, B, N, D, K, dtype, chunk_rows, ctypes.cast(out, ctypes.c_void_p)))
    keys = ("pair", "BN", "XB", "CS", "smem", "Kp", "sort_passes", "sort_block", "update_form")
    return {k: int(v) for k, v in zip(keys, out)}


def ablation_assign_materialized(X: torch.Tensor, C: torch.Tensor, *, chunk_rows: Optional[int] = None,
                                 mindist: bool = True, stream=None):
    """Baseline (not the method): the N x K distance matrix through device
    memory -- a library GEMM writes the scores, an argmin kernel reads them.
    One instance.  Returns (idx int32 [N], mindist float32 [N] or None)."""
    _contig_cuda(X, "X"), _contig_cuda(C, "C")
    if X.dim() != 2 or C.dim() != 2 or C.shape[1] != X.shape[1] or C.dtype != X.dtype:
        raise ValueError("X [N, D] and C [K, D] of one dtype")
    N, D = X.shape
    K = C.shape[0]
    dt = _dtype_code(X)
    _check_tensor(C, "C", X.device)
    _check_stream(stream, X.device)
    cr = N if chunk_rows is None else int(chunk_rows)
    with torch.cuda.device(X.device):
        idx = torch.empty(N, dtype=torch.int32, device=X.device)
        md = torch.empty(N, dtype=torch.float32, device=X.device) if mindist else None
        wsb = int(library().km_ablation_workspace_size(0, N, D, K, dt, cr))
        ws = torch.empty(max(wsb, 1), dtype=torch.uint8, device=X.device)
        _check(library().km_ablation_assign_materialized(_ptr(X), _ptr(C), N, D, K, dt, cr, _ptr(idx), _ptr(md),
                                                         _ptr(ws), ws.numel(), _stream(stream)))
    return idx, md


def ablation_update_atomic(X: torch.Tensor, idx: torch.Tensor, C: torch.Tensor, *, stream=None):
    """Baseline (not the method): every point added to its cluster's sum with
    float atomics, then C = sum / count (empty clusters keep C).  C float32
    [K, D] is updated in place.  Returns counts int32 [K]."""
    _contig_cuda(X, "X"), _contig_cuda(idx, "idx"), _contig_cuda(C, "C")
    if X.dim() != 2 or C.dim() != 2 or C.shape[1] != X.shape[1] or C.dtype != torch.float32:
        raise ValueError("X [N, D] and float32 C [K, D]")
    if idx.dtype != torch.int32 or idx.shape != (X.shape[0],):
        raise ValueError("idx must be int32 [N]")
    N, D = X.shape
    K = C.shape[0]
    dt = _dtype_code(X)
    _check_tensor(idx, "idx", X.device, torch.int32, (N,))
    _check_tensor(C, "C", X.device, torch.float32)
    _check_stream(stream, X.device)
    with torch.cuda.device(X.device):
        counts = torch.empty(K, dtype=torch.int32, device=X.device)
        wsb = int(library().km_ablation_workspace_size(1, N, D, K, dt, 0))
        ws = torch.empty(max(wsb, 1), dtype=torch.uint8, device=X.device)
        _check(library().km_ablation_update_atomic(_ptr(X), _ptr(idx), N, D, K, dt, _ptr(C), _ptr(counts),
                                                   _ptr(ws), ws.numel(), _stream(stream)))
    return counts


def _fit_outputs(X, C0, iters, C_out, idx_out, counts_out, objective, want_idx, stream):
    """Checked shapes and outputs of a fit call (allocated on X's device)."""
    _contig_cuda(X, "X"), _contig_cuda(C0, "C0")
    B, N, D, batched = _shape3(X, "X")
    Bc, K, Dc, _ = _shape3(C0, "C0")
    if Bc != B or Dc != D or C0.dtype != X.dtype:
        raise ValueError("C0 must match X in batch, D and dtype")
    if iters < 0:
        raise ValueError("iters must be >= 0")
    dev = X.device
    _check_tensor(C0, "C0", dev)
    _check_stream(stream, dev)
    cshape, ishape, kshape = ((B, K, D), (B, N), (B, K)) if batched else ((K, D), (N,), (K,))
    oshape = (B, iters) if batched else (iters,)
    if C_out is None:
        C_out = torch.empty(cshape, dtype=torch.float32, device=dev)
    _check_tensor(C_out, "C_out", dev, torch.float32, cshape)
    if idx_out is None and want_idx:
        idx_out = torch.empty(ishape, dtype=torch.int32, device=dev)
    if idx_out is not None:
        _check_tensor(idx_out, "idx_out", dev, torch.int32, ishape)
    if counts_out is None:
        counts_out = torch.empty(kshape, dtype=torch.int32, device=dev)
    _check_tensor(counts_out, "counts_out", dev, torch.int32, kshape)
    if objective is None:
        objective = torch.empty(oshape, dtype=torch.float64, device=dev)
    _check_tensor(objective, "objective", dev, torch.float64, oshape)
    return B, N, D, K, _dtype_code(X), C_out, idx_out, counts_out, objective


def fit(X: torch.Tensor, C0: torch.Tensor, iters: int, *, C_out=None, idx_out=None, counts_out=None,
        objective=None, want_idx: bool = True, workspace=None, stream=None):
    """`iters` exact Lloyd iterations from C0 on the device.

    Returns dict(C float32, idx int32 or None, counts int32, objective float64 [B, iters] or [iters]).
    """
    _contig_cuda(X, "X")
    with torch.cuda.device(X.device):
        B, N, D, K, dt, C_out, idx_out, counts_out, objective = _fit_outputs(
            X, C0, iters, C_out, idx_out, counts_out, objective, want_idx, stream)
        ws = _workspace(OP_FIT, B, N, D, K, dt, X.device, workspace)
        _check_tensor(ws, "workspace", X.device, torch.uint8)
        _check(library().km_fit(_ptr(X), _ptr(C0), B, N, D, K, dt, iters, _ptr(C_out), _ptr(idx_out),
                                _ptr(counts_out), _ptr(objective), _ptr(ws), ws.numel(), _stream(stream)))
    return dict(C=C_out, idx=idx_out, counts=counts_out, objective=objective)


def fit_profile(X: torch.Tensor, C0: torch.Tensor, iters: int, *, C_out=None, idx_out=None, counts_out=None,
                objective=None, workspace=None, stream=None):
    """fit() with CUDA-event timing of each iteration's assignment and update.

    Synchronous.  Returns the fit() dict plus "phase_ms": float32 [iters, 2]
    (assignment kernel ms, update ms) and "iters_ms": device time of the
    iterations (first assignment start to last update end).
    """
    _contig_cuda(X, "X")
    with torch.cuda.device(X.device):
        B, N, D, K, dt, C_out, idx_out, counts_out, objective = _fit_outputs(
            X, C0, iters, C_out, idx_out, counts_out, objective, False, stream)
        phase = torch.zeros(2 * iters + 1, dtype=torch.float32)
        ws = _workspace(OP_FIT, B, N, D, K, dt, X.device, workspace)
        _check_tensor(ws, "workspace", X.device, torch.uint8)
        _check(library().km_fit_profile(_ptr(X), _ptr(C0), B, N, D, K, dt, iters, _ptr(C_out), _ptr(idx_out),
                                        _ptr(counts_out), _ptr(objective), _ptr(ws), ws.numel(), _stream(stream),
                                        _ptr(phase)))
    return dict(C=C_out, idx=idx_out, counts=counts_out, objective=objective,
                phase_ms=phase[:2 * iters].reshape(iters, 2), iters_ms=float(phase[2 * iters]))


def fit_timed(X: torch.Tensor, C0: torch.Tensor, iters: int, *, C_out=None, idx_out=None, counts_out=None,
              objective=None, workspace=None, stream=None):
    """fit() with the device time of its iterations, events around the loop only.

    Synchronous.  Returns the fit() dict plus "iters_ms": device time from
    the first assignment's start to the last update's end.  Unlike
    fit_profile, no event sits between the kernels, so they chain as in fit().
    """
    _contig_cuda(X, "X")
    with torch.cuda.device(X.device):
        B, N, D, K, dt, C_out, idx_out, counts_out, objective = _fit_outputs(
            X, C0, iters, C_out, idx_out, counts_out, objective, False, stream)
        ms = ctypes.c_float(0.0)
        ws = _workspace(OP_FIT, B, N, D, K, dt, X.device, workspace)
        _check_tensor(ws, "workspace", X.device, torch.uint8)
        _check(library().km_fit_timed(_ptr(X), _ptr(C0), B, N, D, K, dt, iters, _ptr(C_out), _ptr(idx_out),
                                      _ptr(counts_out), _ptr(objective), _ptr(ws), ws.numel(), _stream(stream),
                                      ctypes.byref(ms)))
    return dict(C=C_out, idx=idx_out, counts=counts_out, objective=objective, iters_ms=float(ms.value))


class FitGraph:
    """fit() captured once as a CUDA graph (km_fit_graph_create); every
    launch() enqueues one complete fit from C0 into the same output tensors.

    The graph holds pointers: this object keeps X, C0, the outputs and the
    workspace alive, and the caller may refill X / C0 in place between
    launches.  With timed=True, iters_ms() gives the device time of the last
    launch's iterations.  close() (or garbage collection) releases it.
    """

    def __init__(self, X: torch.Tensor, C0: torch.Tensor, iters: int, *, C_out=None, idx_out=None,
                 counts_out=None, objective=None, want_idx: bool = True, workspace=None, timed: bool = False):
        self._h = None
        _contig_cuda(X, "X")
        with torch.cuda.device(X.device):
            B, N, D, K, dt, C_out, idx_out, counts_out, objective = _fit_outputs(
                X, C0, iters, C_out, idx_out, counts_out, objective, want_idx, None)
            ws = _workspace(OP_FIT, B, N, D, K, dt, X.device, workspace)
            _check_tensor(ws, "workspace", X.device, torch.uint8)
            h = ctypes.c_void_p()
            _check(library().km_fit_graph_create(ctypes.byref(h), _ptr(X), _ptr(C0), B, N, D, K, dt, iters,
                                                 _ptr(C_out), _ptr(idx_out), _ptr(counts_out), _ptr(objective),
                                                 _ptr(ws), ws.numel(), 1 if timed else 0))
        self._h = h
        self.device = X.device
        self.X, self.C0, self.workspace = X, C0, ws
        self.result = dict(C=C_out, idx=idx_out, counts=counts_out, objective=objective)

    def launch(self, stream=None) -> dict:
        """Enqueue one fit (asynchronous); returns the output tensors."""
        if self._h is None:
            raise RuntimeError("the graph was closed")
        _check_stream(stream, self.device)
        with torch.cuda.device(self.device):
            _check(library().km_fit_graph_launch(self._h, _stream(stream)))
        return self.result

    def iters_ms(self) -> float:
        """Waits for the last launch; milliseconds of its iterations."""
        ms = ctypes.c_float(0.0)
        _check(library().km_fit_graph_elapsed(self._h, ctypes.byref(ms)))
        return float(ms.value)

    def close(self) -> None:
        if self._h is not None:
            torch.cuda.synchronize(self.device)
            library().km_fit_graph_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def launch_count() -> int:
    """Kernels this library has enqueued in this process so far."""
    return int(library().km_launch_count())


def fit_host(X_host: torch.Tensor, C0: torch.Tensor, iters: int, chunk_rows: int, *, C_out=None, idx_out=None,
             want_idx: bool = False, counts_out=None, workspace=None, stream=None):
    """Out-of-core Lloyd: X_host is a pinned CPU tensor (N, D), streamed per iteration in chunks.

    Synchronous.  Returns dict(C, idx or None, counts, objective (CPU float64 [iters])).
    """
    if X_host.is_cuda or not X_host.is_pinned():
        raise ValueError("X_host must be a pinned CPU tensor")
    if not X_host.is_contiguous():
        raise ValueError("X_host must be contiguous")
    _contig_cuda(C0, "C0")
    if X_host.dim() != 2 or C0.dim() != 2 or C0.shape[1] != X_host.shape[1] or C0.dtype != X_host.dtype:
        raise ValueError("X_host [N, D] and C0 [K, D] of one dtype")
    N, D = X_host.shape
    K = C0.shape[0]
    dt = _dtype_code(X_host)
    dev = C0.device
    _check_stream(stream, dev)
    with torch.cuda.device(dev):
        C_out = torch.empty((K, D), dtype=torch.float32, device=dev) if C_out is None else C_out
        _check_tensor(C_out, "C_out", dev, torch.float32, (K, D))
        if idx_out is None and want_idx:
            idx_out = torch.empty(N, dtype=torch.int32, device=dev)
        if idx_out is not None:
            _check_tensor(idx_out, "idx_out", dev, torch.int32, (N,))
        counts_out = torch.empty(K, dtype=torch.int32, device=dev) if counts_out is None else counts_out
        _check_tensor(counts_out, "counts_out", dev, torch.int32, (K,))
        obj = torch.empty(iters, dtype=torch.float64)
        ws = _workspace(OP_FIT_HOST, 1, N, D, K, dt, dev, workspace, chunk_rows)
        _check_tensor(ws, "workspace", dev, torch.uint8)
        _check(library().km_fit_host(_ptr(X_host), _ptr(C0), N, D, K, dt, iters, chunk_rows, _ptr(C_out),
                                     _ptr(idx_out), _ptr(counts_out), _ptr(obj), _ptr(ws), ws.numel(),
                                     _stream(stream)))
    return dict(C=C_out, idx=idx_out, counts=counts_out, objective=obj)


def fit_source(source, N: int, C0: torch.Tensor, iters: int, chunk_rows: int, *, dtype=torch.bfloat16,
               C_out=None, idx_out=None, want_idx: bool = False, counts_out=None, workspace=None, stream=None):
    """Out-of-core Lloyd over a point set that is never held whole: every
    iteration, source(row0, rows, slot) returns a pinned CPU tensor holding
    rows [row0, row0 + rows) (shape (rows, D), the given dtype).  The tensor
    returned for a slot (0 or 1) is kept alive and unchanged until that slot
    is asked for again.  Same results as fit_host on the concatenated rows.

    Synchronous.  Returns dict(C, idx or None, counts, objective (CPU float64 [iters])).
    """
    _contig_cuda(C0, "C0")
    if C0.dim() != 2 or C0.dtype != dtype:
        raise ValueError("C0 must be [K, D] of the points' dtype")
    K, D = C0.shape
    dt = _dtype_code(C0)
    dev = C0.device
    _check_stream(stream, dev)
    held = [None, None]      # the tensors behind the two slots
    errors = []
    es = C0.element_size()

    def trampoline(_user, row0, rows, slot):
        try:
            t = source(int(row0), int(rows), int(slot))
            if (t.is_cuda or not t.is_pinned() or not t.is_contiguous() or t.dtype != dtype
                    or tuple(t.shape) != (rows, D)):
                raise ValueError(f"the source must return a pinned contiguous {dtype} tensor of shape ({rows}, {D})")
            held[slot] = t
            return t.data_ptr()
        except BaseException as e:  # the library sees NULL and stops
            errors.append(e)
            return None

    cb = CHUNK_SOURCE(trampoline)
    with torch.cuda.device(dev):
        C_out = torch.empty((K, D), dtype=torch.float32, device=dev) if C_out is None else C_out
        _check_tensor(C_out, "C_out", dev, torch.float32, (K, D))
        if idx_out is None and want_idx:
            idx_out = torch.empty(N, dtype=torch.int32, device=dev)
        if idx_out is not None:
            _check_tensor(idx_out, "idx_out", dev, torch.int32, (N,))
        counts_out = torch.empty(K, dtype=torch.int32, device=dev) if counts_out is None else counts_out
        _check_tensor(counts_out, "counts_out", dev, torch.int32, (K,))
        obj = torch.empty(iters, dtype=torch.float64)
        ws = _workspace(OP_FIT_HOST, 1, N, D, K, dt, dev, workspace, chunk_rows)
        _check_tensor(ws, "workspace", dev, torch.uint8)
        st = library().km_fit_source(cb, None, _ptr(C0), N, D, K, dt, iters, chunk_rows, _ptr(C_out),
                                     _ptr(idx_out), _ptr(counts_out), _ptr(obj), _ptr(ws), ws.numel(),
                                     _stream(stream))
    if errors:
        raise errors[0]
    _check(st)
    del es
    return dict(C=C_out, idx=idx_out, counts=counts_out, objective=obj)


def workspace_status(workspace: torch.Tensor, stream=None) -> int:
    """Synchronise and read/clear the workspace status word (0 or KM_ERR_TIMEOUT)."""
    return int(library().km_workspace_status(_ptr(workspace), _stream(stream)))


def selftest_timeout(limit_ns: int = 1_000_000, device="cuda") -> int:
    """Run the bounded-wait self-test kernel; returns the status it reports."""
    ws = torch.zeros(256, dtype=torch.uint8, device=device)
    return int(library().km_selftest_timeout(_ptr(ws), ws.numel(), int(limit_ns), _stream(None)))


# ------------------------------------------------------------ soft assignment
class Quantized(NamedTuple):
    """Points in 8 bits: data float8_e4m3fn (..., N, D), rows ceil(D / 16) * 16
    bytes apart, and scale float8_e8m0fnu (..., N, ceil(D / 128)), one power of
    two per 128 coordinates; coordinate d stands for data[d] * scale[d // 128]."""
    data: torch.Tensor
    scale: torch.Tensor


class Balance(NamedTuple):
    """What balance() returns: the loss float32 [B], the picks per cluster int32
    (K,) or (B, K), and what its gradient needs: the valid points int32 [B], each
    row's logsumexp and sum of p * (K * share - 1) float32 (N,) or (B, N), and the
    picks per point."""
    loss: torch.Tensor
    counts: torch.Tensor
    rows: torch.Tensor
    lse: torch.Tensor
    dot: torch.Tensor
    picks: int


@functools.lru_cache(maxsize=4096)
def soft_workspace_size(op: int, B: int, N: int, D: int, K: int, dtype: int) -> int:
    n = library().km_soft_workspace_size(op, B, N, D, K, dtype)
    if n == 0:
        raise KMError(2, library().km_last_error().decode(errors="replace"))
    return int(n)


class _on:
    """Device and stream of a call: outputs and workspaces allocated inside
    belong to the stream the kernels run on, and .raw is that stream.  Nothing
    is switched where the caller's device and stream are meant: the calls of a
    training or serving loop take microseconds."""

    __slots__ = ("_d", "_s", "raw")

    def __init__(self, device, stream):
        if stream is not None and stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the points are on {device}")
        self._d = None if device.index == torch._C._cuda_getDevice() else torch.cuda.device(device)
        self._s = None if stream is None else torch.cuda.stream(stream)
        self.raw = torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream

    def __enter__(self):
        if self._d is not None:
            self._d.__enter__()
        if self._s is not None:
            self._s.__enter__()
        return self.raw

    def __exit__(self, *a):
        if self._s is not None:
            self._s.__exit__(*a)
        if self._d is not None:
            self._d.__exit__(*a)


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _soft_workspace(op, B, N, D, K, dtype, device, workspace):
    need = soft_workspace_size(op, B, N, D, K, dtype)
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    _check_tensor(workspace, "workspace", device, torch.uint8)
    if workspace.numel() < need:
        raise ValueError(f"workspace has {workspace.numel()} bytes, needs {need}")
    return workspace


_status_words = {}


def _scores_workspace(B, N, D, K, dtype, device, raw, workspace):
    """scores() needs a workspace for its status word alone, which nobody reads
    where the caller brings none: one for each device and stream serves all such
    calls.  (Not one for all streams: memory is in order on the stream it was
    allocated on, and another's call could clear it while work queued there
    before still uses it.)  A captured call takes its graph's memory, since the
    graph may be replayed on any stream."""
    if workspace is not None:
        return _soft_workspace(SOFT_SCORES, B, N, D, K, dtype, device, workspace)
    captured = torch.cuda.is_current_stream_capturing()
    ws = None if captured else _status_words.get((device.index, raw))
    if ws is None:   # of one size for every shape
        ws = torch.empty(soft_workspace_size(SOFT_SCORES, B, N, D, K, dtype), dtype=torch.uint8, device=device)
        if not captured:
            _status_words[device.index, raw] = ws
    return ws


def _soft_dtype(dtype) -> int:
    if dtype == torch.bfloat16:
        return BF16
    if dtype == torch.float32:
        return F32
    raise TypeError(f"the type must be bfloat16 or float32, got {dtype}")


def _new_quantized(lead, D, device) -> Quantized:
    ld = (D + 15) // 16 * 16
    data = torch.empty(*lead, ld, dtype=torch.float8_e4m3fn, device=device)
    scale = torch.empty(*lead, (D + 127) // 128, dtype=torch.float8_e8m0fnu, device=device)
    return Quantized(data if ld == D else data[..., :D], scale)


def _check_quantized(q, name: str, device=None):
    """Shape (B, N, D, batched) of 8-bit points, their layout checked: dense
    rows ceil(D / 16) * 16 bytes apart and dense scales of the same points."""
    if not isinstance(q, tuple) or len(q) != 2:
        raise TypeError(f"{name} must be Quantized (data, scale)")
    data, scale = q
    if not data.is_cuda or not scale.is_cuda:
        raise ValueError(f"{name} must be CUDA tensors")
    if data.dtype != torch.float8_e4m3fn or scale.dtype != torch.float8_e8m0fnu:
        raise TypeError(f"{name} must be float8_e4m3fn data and float8_e8m0fnu scale, got {data.dtype}, {scale.dtype}")
    B, N, D, batched = _shape3(data, name)
    ld = (D + 15) // 16 * 16
    want = ((N * ld, ld, 1) if batched else (ld, 1))
    if data.stride() != want and any(n > 1 and s != w for n, s, w in zip(data.shape, data.stride(), want)):
        raise ValueError(f"rows of {name}.data must be dense and {ld} bytes apart")
    if data.data_ptr() % 16 and data.numel():
        raise ValueError(f"{name}.data must be 16-byte aligned")
    if ld != D and data.numel() and data.untyped_storage().nbytes() - data.storage_offset() < B * N * ld:
        raise ValueError(f"the last row of {name}.data must have {ld} bytes")
    dev = data.device
    _check_tensor(scale, f"{name}.scale", dev, None, (*data.shape[:-1], (D + 127) // 128))
    if device is not None and dev != device:
        raise ValueError(f"{name} is on {dev}, the points are on {device}")
    return B, N, D, batched


def quantize(X: torch.Tensor, *, out: Optional[Quantized] = None, stream=None) -> Quantized:
    """Points (N, D) or (B, N, D), bf16 or f32, kept in 8 bits: half or a quarter
    of the bytes between a forward and a backward pass, and the operand of
    scores() and scores_grad().  See km_quantize for the rounding."""
    _contig_cuda(X, "X")
    B, N, D, _ = _shape3(X, "X")
    dt = _dtype_code(X)
    dev = X.device
    with _on(dev, stream) as raw:
        if out is None:
            out = _new_quantized(X.shape[:-1], D, dev)
        else:
            if out.data.shape != X.shape:
                raise ValueError(f"out must have shape {tuple(X.shape)}, got {tuple(out.data.shape)}")
            _check_quantized(out, "out", dev)
        _check(library().km_quantize(X.data_ptr(), B, N, D, dt, out.data.data_ptr(), out.scale.data_ptr(), raw))
    return out


def dequantize(q: Quantized, dtype: torch.dtype = torch.bfloat16, *, out=None, stream=None) -> torch.Tensor:
    """The values 8-bit points stand for, in bf16 or f32 (exact in both)."""
    B, N, D, _ = _check_quantized(q, "q")
    dt = _soft_dtype(dtype)
    data, scale = q
    dev = data.device
    with _on(dev, stream) as raw:
        if out is None:
            out = torch.empty(data.shape, dtype=dtype, device=dev)
        else:
            _check_tensor(out, "out", dev, dtype, data.shape)
        _check(library().km_dequantize(data.data_ptr(), scale.data_ptr(), B, N, D, dt, out.data_ptr(), raw))
    return out


def _score_args(X, C):
    B, N, D, batched = _check_quantized(X, "X")
    dev = X.data.device
    Bc, K, Dc, batched_c = _check_quantized(C, "C", dev)
    if Bc != B or Dc != D or batched_c != batched:
        raise ValueError("C must match X in batch and D")
    return B, N, D, K, batched, dev


def scores(X: Quantized, C: Quantized, *, bias: Optional[torch.Tensor] = None, alpha: float = 1.0,
           dtype: torch.dtype = torch.float32, out=None, workspace=None, stream=None) -> torch.Tensor:
    """Scores of 8-bit points against 8-bit centroids: bias + alpha * x . c for
    every pair, (N, K) or (B, N, K) in `dtype` (bf16 or f32).  bias float32 (K,)
    or (B, K).  alpha = 2 / t and bias = -|c|^2 / t give the logits of a soft
    assignment by distance.  As with assign(), workspace_status() of a workspace
    passed in tells of an in-kernel wait that ran out."""
    B, N, D, K, batched, dev = _score_args(X, C)
    dt = _soft_dtype(dtype)
    shp = (B, N, K) if batched else (N, K)
    if bias is not None:
        _check_tensor(bias, "bias", dev, torch.float32, (B, K) if batched else (K,))
    with _on(dev, stream) as raw:
        if out is None:
            out = torch.empty(shp, dtype=dtype, device=dev)
        else:
            _check_tensor(out, "out", dev, dtype, shp)
        ws = _scores_workspace(B, N, D, K, dt, dev, raw, workspace)
        _check(library().km_scores(X.data.data_ptr(), X.scale.data_ptr(), C.data.data_ptr(), C.scale.data_ptr(),
                                   _addr(bias), alpha, B, N, D, K, dt, out.data_ptr(), ws.data_ptr(), ws.numel(), raw))
    return out


def scores_grad(dS: torch.Tensor, X: Quantized, C: Quantized, *, alpha: float = 1.0,
                dtype: Optional[torch.dtype] = None, want_dX: bool = True, want_dC: bool = True,
                want_dbias: bool = True, workspace=None, stream=None):
    """Gradients of scores() for the gradient dS (bf16 or f32) of its result,
    with respect to the values the 8-bit X and C stand for.  dS starts on a
    16-byte boundary, as a tensor of its own does (a view of an odd offset may not).

    Returns (dX in `dtype`, by default dS's, dC float32, dbias float32), None for
    those not wanted."""
    _contig_cuda(dS, "dS")
    B, N, D, K, batched, dev = _score_args(X, C)
    _check_tensor(dS, "dS", dev, None, (B, N, K) if batched else (N, K))
    dt = _dtype_code(dS)
    dtype = dS.dtype if dtype is None else dtype
    dxt = _soft_dtype(dtype)
    if not (want_dX or want_dC or want_dbias):
        raise ValueError("one of dX, dC and dbias must be wanted")
    lead = (B,) if batched else ()
    with _on(dev, stream) as raw:
        dX = torch.empty((*lead, N, D), dtype=dtype, device=dev) if want_dX else None
        dC = torch.empty((*lead, K, D), dtype=torch.float32, device=dev) if want_dC else None
        db = torch.empty((*lead, K), dtype=torch.float32, device=dev) if want_dbias else None
        ws = _soft_workspace(SOFT_SCORES_GRAD, B, N, D, K, dt, dev, workspace)
        _check(library().km_scores_grad(dS.data_ptr(), X.data.data_ptr(), X.scale.data_ptr(), C.data.data_ptr(),
                                        C.scale.data_ptr(), alpha, B, N, D, K, dt, dxt, _addr(dX), _addr(dC), _addr(db),
                                        ws.data_ptr(), ws.numel(), raw))
    return dX, dC, db


def _valid_mask(valid, shape, device):
    if valid is None:
        return None
    if valid.dtype not in (torch.bool, torch.uint8):
        raise ValueError(f"valid must be bool or uint8, got {valid.dtype}")
    return _check_tensor(valid, "valid", device, None, shape)


def balance(S: torch.Tensor, idx: torch.Tensor, *, valid: Optional[torch.Tensor] = None, workspace=None,
            stream=None) -> Balance:
    """Balance loss of the soft assignment softmax(S) under the picks idx, and
    the picks per cluster.  S (N, K) or (B, N, K) bf16/f32; idx int32 (N,) or
    (B, N), or with T picks per point (N, T) or (B, N, T); valid (N,) or (B, N)
    bool: the points that count.  S starts on a 16-byte boundary, as a tensor of its
    own does; at most 1024 picks per point.  See km_balance."""
    _contig_cuda(S, "S")
    B, N, K, batched = _shape3(S, "S")
    dt = _dtype_code(S)
    dev = S.device
    lead = (B, N) if batched else (N,)
    many = idx.dim() == len(lead) + 1
    T = idx.shape[-1] if many else 1
    if T < 1:
        raise ValueError("idx must hold at least one pick per point")
    _check_tensor(idx, "idx", dev, torch.int32, (*lead, T) if many else lead)
    valid = _valid_mask(valid, lead, dev)
    with _on(dev, stream) as raw:
        loss = torch.empty(B, dtype=torch.float32, device=dev)
        counts = torch.empty((B, K) if batched else (K,), dtype=torch.int32, device=dev)
        rows = torch.empty(B, dtype=torch.int32, device=dev)
        lse = torch.empty(lead, dtype=torch.float32, device=dev)
        dot = torch.empty(lead, dtype=torch.float32, device=dev)
        ws = _soft_workspace(SOFT_BALANCE, B, N, 1, K, dt, dev, workspace)
        _check(library().km_balance(S.data_ptr(), idx.data_ptr(), _addr(valid), B, N, K, T, dt, loss.data_ptr(),
                                    counts.data_ptr(), rows.data_ptr(), lse.data_ptr(), dot.data_ptr(), ws.data_ptr(),
                                    ws.numel(), raw))
    return Balance(loss, counts, rows, lse, dot, T)


def balance_grad(S: torch.Tensor, bal: Balance, *, grad: Optional[torch.Tensor] = None,
                 valid: Optional[torch.Tensor] = None, out=None, stream=None) -> torch.Tensor:
    """Gradient of balance()'s loss with respect to S (S's type), given what
    balance() returned for the same S and valid; grad float32 [B] is the
    gradient of the loss itself (1 if not given)."""
    _contig_cuda(S, "S")
    B, N, K, batched = _shape3(S, "S")
    dt = _dtype_code(S)
    dev = S.device
    lead = (B, N) if batched else (N,)
    _check_tensor(bal.counts, "counts", dev, torch.int32, (B, K) if batched else (K,))
    _check_tensor(bal.rows, "rows", dev, torch.int32, (B,))
    _check_tensor(bal.lse, "lse", dev, torch.float32, lead)
    _check_tensor(bal.dot, "dot", dev, torch.float32, lead)
    valid = _valid_mask(valid, lead, dev)
    if grad is not None:
        _check_tensor(grad, "grad", dev, torch.float32, (B,))
    with _on(dev, stream) as raw:
        if out is None:
            out = torch.empty_like(S)
        else:
            _check_tensor(out, "out", dev, S.dtype, S.shape)
            if out.numel() and abs(out.data_ptr() - S.data_ptr()) < S.numel() * S.element_size():
                raise ValueError("out must not overlap S")
        _check(library().km_balance_grad(S.data_ptr(), _addr(valid), bal.counts.data_ptr(), bal.rows.data_ptr(),
                                         bal.lse.data_ptr(), bal.dot.data_ptr(), _addr(grad), B, N, K, bal.picks, dt,
                                         out.data_ptr(), raw))
    return out
