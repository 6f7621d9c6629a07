"""Python binding of neighbour attention and the distance buckets (include/tp_attn.h): argument
marshalling only; every step runs in libtp.so.

Tensors of one call lie on one device; the call runs there, whatever the current device is, on
that device's current stream or on `stream`.  Outputs and workspaces that a call makes itself are
allocated for the stream that it runs on.
"""
from __future__ import annotations

import ctypes as C
import math
from typing import Optional

import torch

from ._lib import TP_OP_BWD, TP_OP_FWD, check, load
from ._marshal import apart, device_index, f32, on, ptr, rows, stream_of, workspace

_I32, _I64, _F32 = torch.int32, torch.int64, torch.float32

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
        self._sizes = {}

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value:
            self._lib.tp_attn_destroy(h)
            self.handle = None


def tp_attn_workspace_size(attn: Attention, N: int, E: int, op: int) -> int:
    out = C.c_size_t()
    check(load().tp_attn_workspace_size(attn.handle, int(N), int(E), int(op), C.byref(out)), "tp_attn_workspace_size")
    return out.value


def _workspace_size(attn, N, E, op):
    """tp_attn_workspace_size, asked once for calls of the same size in a row."""
    last = attn._sizes.get(op)
    if last is None or last[0] != N or last[1] != E:
        last = attn._sizes[op] = (N, E, tp_attn_workspace_size(attn, N, E, op))
    return last[2]


def _inputs(attn, rowptr, src, q, k, v, bucket, table, scale, p, rng, site):
    N, E, qk = rowptr.numel() - 1, src.numel(), attn.qk_dim
    if N < 0:
        raise ValueError("rowptr must have N + 1 entries")
    if q.shape != (N, qk) or k.shape != (N, qk) or v.shape != (N, attn.v_dim):
        raise ValueError(f"q, k, v must have shapes {[N, qk]}, {[N, qk]}, {[N, attn.v_dim]}, got "
                         f"{list(q.shape)}, {list(k.shape)}, {list(v.shape)}")
    if bucket is not None and bucket.shape != (E,):
        raise ValueError(f"bucket must have shape {[E]}, got {list(bucket.shape)}")
    if table is not None and table.shape != (attn.n_buckets, attn.heads):
        raise ValueError(f"table must have shape {[attn.n_buckets, attn.heads]}, got {list(table.shape)}")
    i = device_index(q, "q")
    if scale is None:
        scale = math.sqrt(attn.heads / qk)
    q, ldq = rows(q, i, N, qk, "q")
    k, ldk = rows(k, i, N, qk, "k")
    v, ldv = rows(v, i, N, attn.v_dim, "v")
    return N, E, i, (ptr(rowptr, _I32, i, None, "rowptr"), ptr(src, _I32, i, None, "src")), (
        ptr(bucket, _I32, i, None, "bucket"), q, ldq, k, ldk, v, ldv, f32(table, i, None, "table"), float(scale), float(p),
        ptr(rng, _I64, i, (2,), "rng"), int(site))


def _pointers(args):
    """bucket, q, k, v, table and rng of what _inputs returns."""
    return args[0], args[1], args[3], args[5], args[7], args[10]


def tp_attn_fwd(attn: Attention, rowptr, src, q, k, v, bucket=None, table=None, scale: Optional[float] = None,
                p: float = 0.0, rng=None, site: int = 0, y=None, lse=None, need_lse: bool = True, ws=None,
                stream=None):
    """(y [N, v_dim], lse [N, heads]); lse is None when need_lse is False.  scale: default
    1/sqrt(floats of a head of q).  p > 0 drops probabilities with rng = int64 CUDA tensor (seed, offset).  y, lse
    and ws may not share memory with an input."""
    N, E, i, graph, args = _inputs(attn, rowptr, src, q, k, v, bucket, table, scale, p, rng, site)
    given = y is not None or lse is not None or ws is not None
    with on(i, stream):
        dev = q.device
        if y is None:
            y = torch.empty(N, attn.v_dim, dtype=_F32, device=dev)
        if lse is None and need_lse:
            lse = torch.empty(N, attn.heads, dtype=_F32, device=dev)
        ws, ws_ptr, ws_bytes = workspace(ws, _workspace_size(attn, N, E, TP_OP_FWD), i)
        out = f32(y, i, (N, attn.v_dim), "y"), f32(lse, i, (N, attn.heads), "lse")
        if given:
            apart((*out, ws_ptr), (*graph, *_pointers(args)), "y, lse and the workspace")
        check(attn._lib.tp_attn_fwd(attn.handle, N, E, *graph, *args, *out, ws_ptr, ws_bytes, stream_of(i)), "tp_attn_fwd")
    return y, lse


def tp_attn_bwd(attn: Attention, rowptr, src, q, k, v, y, lse, gy, bucket=None, table=None,
                scale: Optional[float] = None, p: float = 0.0, rng=None, site: int = 0, colptr=None, perm=None,
                need_gq=True, need_gk=True, need_gv=True, need_gtable: Optional[bool] = None, gq=None, gk=None,
                gv=None, gtable=None, ws=None, stream=None):
    """(gq, gk, gv, gtable) against gy, each None when not requested; y and lse from tp_attn_fwd with the same
    arguments.  need_gtable: default whenever there is a table.  gq, gk, gv may be column slices, but share no
    memory with an input or one another."""
    if (colptr is None) != (perm is None):
        raise ValueError("colptr and perm must both be given or both be None")
    N, E, i, graph, args = _inputs(attn, rowptr, src, q, k, v, bucket, table, scale, p, rng, site)
    if need_gtable is None:
        need_gtable = table is not None or gtable is not None
    qk, vd = attn.qk_dim, attn.v_dim
    table_shape = (attn.n_buckets, attn.heads)
    given = any(t is not None for t in (gq, gk, gv, gtable, ws))
    with on(i, stream):
        dev = q.device
        gq = torch.empty(N, qk, dtype=_F32, device=dev) if gq is None and need_gq else gq
        gk = torch.empty(N, qk, dtype=_F32, device=dev) if gk is None and need_gk else gk
        gv = torch.empty(N, vd, dtype=_F32, device=dev) if gv is None and need_gv else gv
        gtable = torch.empty(table_shape, dtype=_F32, device=dev) if gtable is None and need_gtable else gtable
        ws, ws_ptr, ws_bytes = workspace(ws, _workspace_size(attn, N, E, TP_OP_BWD), i)
        order = ptr(colptr, _I32, i, (N + 1,), "colptr"), ptr(perm, _I32, i, (E,), "perm")
        saved = f32(y, i, (N, vd), "y"), f32(lse, i, (N, attn.heads), "lse"), f32(gy, i, (N, vd), "gy")
        out = (*rows(gq, i, N, qk, "gq"), *rows(gk, i, N, qk, "gk"), *rows(gv, i, N, vd, "gv"),
               f32(gtable, i, table_shape, "gtable"))
        if given:
            apart((*out[::2], ws_ptr), (*graph, *order, *_pointers(args), *saved), "gq, gk, gv, gtable and the workspace")
        check(attn._lib.tp_attn_bwd(attn.handle, N, E, *graph, *order, *args, *saved, *out, ws_ptr, ws_bytes, stream_of(i)),
              "tp_attn_bwd")
    return gq, gk, gv, gtable


def tp_distance_buckets(vec, bounds, cutoff: Optional[float] = None, bucket=None, stream=None):
    """int32 [E]: how many of the ascending bounds are <= |vec[e]|, or -1 from the cutoff on (and for NaN)."""
    E = vec.shape[0]
    if vec.shape != (E, 3):
        raise ValueError(f"vec must have shape [E, 3], got {list(vec.shape)}")
    i, n = device_index(vec, "vec"), bounds.numel()
    with on(i, stream):
        if bucket is None:
            bucket = torch.empty(E, dtype=_I32, device=vec.device)
        check(load().tp_distance_buckets(E, f32(vec, i, None, "vec"), n, f32(bounds, i, (n,), "bounds"),
                                         math.inf if cutoff is None else float(cutoff), ptr(bucket, _I32, i, (E,), "bucket"),
                                         stream_of(i)), "tp_distance_buckets")
    return bucket
