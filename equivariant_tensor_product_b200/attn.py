"""Python binding of neighbour attention and the distance buckets (include/tp_attn.h): argument
marshalling only; every step runs in libtp.so.

Tensors of one call lie on one device; the call runs there, whatever the current device is, on
that device's current stream or on `stream`.  Outputs and workspaces that a call makes itself are
allocated for the stream that it runs on.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import math
from typing import Optional

import torch

from ._lib import TP_OP_BWD, TP_OP_FWD, check, load
from .ops import _ptr

__all__ = ["Attention", "tp_attn_fwd", "tp_attn_bwd", "tp_attn_workspace_size", "tp_distance_buckets"]


class Attention:
    """Owns a tp_attn_t: softmax attention over each receiver's edges, `heads` heads over the channels of
    every block, with a bias table of n_buckets rows (0: no buckets)."""

    def __init__(self, irreps_qk: str, irreps_v: str, heads: int, n_buckets: int = 0):
        lib = load()
        self._lib = lib
        self.handle = C.c_void_p()
        self.irreps_qk, self.irreps_v = irreps_qk, irreps_v
        self.heads, self.n_buckets = int(heads), int(n_buckets)
        check(lib.tp_attn_create(C.byref(self.handle), irreps_qk.encode(), irreps_v.encode(), self.heads,
                                 self.n_buckets), "tp_attn_create")
        a, b = C.c_int64(), C.c_int64()
        check(lib.tp_attn_query(self.handle, C.byref(a), C.byref(b)), "tp_attn_query")
        self.qk_dim, self.v_dim = a.value, b.value

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value:
            self._lib.tp_attn_destroy(h)
            self.handle = None


def _on(device, stream):
    """The context a call runs in: `device` current and, when given, `stream` its current stream."""
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a CUDA device, got {device}")
    if stream is None:
        if torch.cuda.current_device() == device.index:
            return contextlib.nullcontext()
        return torch.cuda.device(device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    elif stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return torch.cuda.stream(stream)


def _same_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} must be on {device}, got {t.device}")


def _shape(t, shape, name):
    if t is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")


def _rows(t, n, width, name):
    """Pointer and row stride of an [n, width] fp32 tensor whose rows are contiguous (a column slice of a
    wider array is fine)."""
    if t is None:
        return None, width
    _shape(t, (n, width), name)
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.float32:
        raise ValueError(f"{name} must be {torch.float32}, got {t.dtype}")
    ld = t.stride(0) if n > 1 else width
    if (width > 1 and t.stride(1) != 1) or ld < width:
        raise ValueError(f"{name} must have contiguous rows at least {width} floats apart")
    return (t.data_ptr() if n else None), ld


def _workspace(ws, need, device):
    if ws is None:
        return torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    if ws.numel() * ws.element_size() < need:
        raise ValueError(f"workspace needs {need} bytes, got {ws.numel() * ws.element_size()}")
    return ws


def tp_attn_workspace_size(attn: Attention, N: int, E: int, op: int) -> int:
    out = C.c_size_t()
    check(load().tp_attn_workspace_size(attn.handle, int(N), int(E), int(op), C.byref(out)), "tp_attn_workspace_size")
    return out.value


def _inputs(attn, rowptr, src, q, k, v, bucket, table, scale, p, rng, site):
    N, E, dev = rowptr.numel() - 1, src.numel(), q.device
    if N < 0:
        raise ValueError("rowptr must have N + 1 entries")
    _same_device(dev, rowptr=rowptr, src=src, k=k, v=v, bucket=bucket, table=table, rng=rng)
    for t, width, name in ((q, attn.qk_dim, "q"), (k, attn.qk_dim, "k"), (v, attn.v_dim, "v")):
        _shape(t, (N, width), name)
    _shape(bucket, (E,), "bucket")
    _shape(table, (attn.n_buckets, attn.heads), "table")
    _shape(rng, (2,), "rng")
    if scale is None:
        scale = math.sqrt(attn.heads / attn.qk_dim)
    args = (_ptr(bucket, torch.int32, "bucket"), *_rows(q, N, attn.qk_dim, "q"), *_rows(k, N, attn.qk_dim, "k"),
            *_rows(v, N, attn.v_dim, "v"), _ptr(table, torch.float32, "table"), float(scale), float(p),
            _ptr(rng, torch.int64, "rng"), int(site))
    return N, E, dev, args


def tp_attn_fwd(attn: Attention, rowptr, src, q, k, v, bucket=None, table=None, scale: Optional[float] = None,
                p: float = 0.0, rng=None, site: int = 0, y=None, lse=None, need_lse: bool = True, ws=None,
                stream=None):
    """(y [N, v_dim], lse [N, heads]); lse is None when need_lse is False.  scale: default
    1/sqrt(floats of a head of q).  p > 0 drops probabilities with rng = int64 CUDA tensor (seed, offset)."""
    N, E, dev, args = _inputs(attn, rowptr, src, q, k, v, bucket, table, scale, p, rng, site)
    _same_device(dev, y=y, lse=lse, ws=ws)
    _shape(y, (N, attn.v_dim), "y")
    _shape(lse, (N, attn.heads), "lse")
    with _on(dev, stream):
        if y is None:
            y = torch.empty(N, attn.v_dim, dtype=torch.float32, device=dev)
        if lse is None and need_lse:
            lse = torch.empty(N, attn.heads, dtype=torch.float32, device=dev)
        ws = _workspace(ws, tp_attn_workspace_size(attn, N, E, TP_OP_FWD), dev)
        check(load().tp_attn_fwd(attn.handle, N, E, _ptr(rowptr, torch.int32, "rowptr"),
                                 _ptr(src, torch.int32, "src"), *args, _ptr(y, torch.float32, "y"),
                                 _ptr(lse, torch.float32, "lse"), ws.data_ptr(), ws.numel() * ws.element_size(),
                                 torch.cuda.current_stream(dev).cuda_stream), "tp_attn_fwd")
    return y, lse


def tp_attn_bwd(attn: Attention, rowptr, src, q, k, v, y, lse, gy, bucket=None, table=None,
                scale: Optional[float] = None, p: float = 0.0, rng=None, site: int = 0, colptr=None, perm=None,
                need_gq=True, need_gk=True, need_gv=True, need_gtable: Optional[bool] = None, gq=None, gk=None,
                gv=None, gtable=None, ws=None, stream=None):
    """(gq, gk, gv, gtable) against gy, each None when not requested; y and lse from tp_attn_fwd with the same
    arguments.  need_gtable: default whenever there is a table.  gq, gk, gv may be column slices."""
    if (colptr is None) != (perm is None):
        raise ValueError("colptr and perm must both be given or both be None")
    N, E, dev, args = _inputs(attn, rowptr, src, q, k, v, bucket, table, scale, p, rng, site)
    _same_device(dev, y=y, lse=lse, gy=gy, colptr=colptr, perm=perm, gq=gq, gk=gk, gv=gv, gtable=gtable, ws=ws)
    for t, shape, name in ((y, (N, attn.v_dim), "y"), (lse, (N, attn.heads), "lse"), (gy, (N, attn.v_dim), "gy"),
                           (gtable, (attn.n_buckets, attn.heads), "gtable"), (colptr, (N + 1,), "colptr"),
                           (perm, (E,), "perm")):
        _shape(t, shape, name)
    if need_gtable is None:
        need_gtable = table is not None or gtable is not None
    with _on(dev, stream):
        new = lambda *shape: torch.empty(*shape, dtype=torch.float32, device=dev)
        gq = new(N, attn.qk_dim) if gq is None and need_gq else gq
        gk = new(N, attn.qk_dim) if gk is None and need_gk else gk
        gv = new(N, attn.v_dim) if gv is None and need_gv else gv
        gtable = new(attn.n_buckets, attn.heads) if gtable is None and need_gtable else gtable
        ws = _workspace(ws, tp_attn_workspace_size(attn, N, E, TP_OP_BWD), dev)
        check(load().tp_attn_bwd(attn.handle, N, E, _ptr(rowptr, torch.int32, "rowptr"),
                                 _ptr(src, torch.int32, "src"), _ptr(colptr, torch.int32, "colptr"),
                                 _ptr(perm, torch.int32, "perm"), *args, _ptr(y, torch.float32, "y"),
                                 _ptr(lse, torch.float32, "lse"), _ptr(gy, torch.float32, "gy"),
                                 *_rows(gq, N, attn.qk_dim, "gq"), *_rows(gk, N, attn.qk_dim, "gk"),
                                 *_rows(gv, N, attn.v_dim, "gv"), _ptr(gtable, torch.float32, "gtable"),
                                 ws.data_ptr(), ws.numel() * ws.element_size(),
                                 torch.cuda.current_stream(dev).cuda_stream), "tp_attn_bwd")
    return gq, gk, gv, gtable


def tp_distance_buckets(vec, bounds, cutoff: Optional[float] = None, bucket=None, stream=None):
    """int32 [E]: how many of the ascending bounds are <= |vec[e]|, or -1 from the cutoff on (and for NaN)."""
    E, dev = vec.shape[0], vec.device
    _shape(vec, (E, 3), "vec")
    _shape(bounds, (bounds.numel(),), "bounds")
    _shape(bucket, (E,), "bucket")
    _same_device(dev, bounds=bounds, bucket=bucket)
    vec_ptr, bounds_ptr = _ptr(vec, torch.float32, "vec"), _ptr(bounds, torch.float32, "bounds")
    with _on(dev, stream):
        if bucket is None:
            bucket = torch.empty(E, dtype=torch.int32, device=dev)
        check(load().tp_distance_buckets(E, vec_ptr, bounds.numel(), bounds_ptr,
                                         math.inf if cutoff is None else float(cutoff),
                                         _ptr(bucket, torch.int32, "bucket"),
                                         torch.cuda.current_stream(dev).cuda_stream), "tp_distance_buckets")
    return bucket
