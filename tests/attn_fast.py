"""The attention of oracle/attn.py over whole edge lists at once, for graphs that its loops over receivers are
too slow for: float64, the formulas of the backward pass written out, pinned against the loops in
tests/test_attn_fast.py."""
from __future__ import annotations

import numpy as np
import torch

from oracle.attn import head_columns


def keep_values(seed, offset, n, p):
    """oracle.attn.keep_values in 64-bit unsigned arrays."""
    u, mask, half = np.uint64, np.uint64(0xFFFFFFFF), np.uint64(32)
    block = np.arange((n + 3) // 4, dtype=u)
    fill = lambda a: np.full_like(block, a & 0xFFFFFFFF)
    c = [block & mask, block >> half, fill(offset), fill(offset >> 32)]
    k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        a, b = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(b >> half) ^ c[1] ^ u(k[0]), b & mask, (a >> half) ^ c[3] ^ u(k[1]), a & mask]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.where(np.stack(c, 1).reshape(-1)[:n] >= u(round(p * 2.0 ** 32)), 1.0 / (1.0 - p), 0.0)


def attention_backward(irreps_qk, irreps_v, heads, rowptr, src, q, k, v, gy, bucket=None, table=None, n_buckets=0, scale=1.0,
                       r=None):
    """{"y", "lse", "gq", "gk", "gv", "gtable"}, rowptr[0] = 0."""
    rowptr = np.asarray(rowptr, np.int64)
    N, E = len(rowptr) - 1, int(rowptr[-1])
    dst, src = np.repeat(np.arange(N), np.diff(rowptr)), np.asarray(src)[:E]
    live = (src >= 0) & (src < N)
    if bucket is not None:
        bucket = np.asarray(bucket)[:E]
        live &= (bucket >= 0) & (bucket < n_buckets)
    f = lambda a: np.asarray(a, np.float64)
    q, k, v, gy = f(q), f(k), f(v), f(gy)
    out = dict(y=np.zeros_like(v), lse=np.full((N, heads), -np.inf), gq=np.zeros_like(q), gk=np.zeros_like(k), gv=np.zeros_like(v))
    if table is not None:
        out["gtable"] = np.zeros((n_buckets, heads))
    for h, (cq, cv) in enumerate(zip(head_columns(irreps_qk, heads), head_columns(irreps_v, heads))):
        e = np.nonzero(live if table is None else live & (f(table)[np.where(live, bucket, 0), h] != -np.inf))[0]
        i, j = dst[e], src[e]
        s = scale * np.einsum("ec,ec->e", q[i][:, cq], k[j][:, cq])
        if table is not None:
            s = s + f(table)[bucket[e], h]
        top = np.full(N, -np.inf)
        np.maximum.at(top, i, s)
        w = np.exp(s - top[i])
        total = np.bincount(i, w, N)
        with np.errstate(divide="ignore"):
            out["lse"][:, h] = np.where(total > 0, top + np.log(total), -np.inf)
        p = w / total[i]
        pr = p if r is None else p * np.asarray(r)[e, h]
        g, vj, kj, qi = gy[i][:, cv], v[j][:, cv], k[j][:, cq], q[i][:, cq]

        def add(name, at, cols, values):
            t = np.zeros((N, len(cols)))
            np.add.at(t, at, values)
            out[name][:, cols] = t
        add("y", i, cv, pr[:, None] * vj)
        delta = (gy[:, cv] * out["y"][:, cv]).sum(1)
        ds = pr * (g * vj).sum(1) - p * delta[i]
        add("gq", i, cq, scale * ds[:, None] * kj)
        add("gk", j, cq, scale * ds[:, None] * qi)
        add("gv", j, cv, pr[:, None] * g)
        if table is not None:
            out["gtable"][:, h] = np.bincount(bucket[e], ds, n_buckets)
    return {name: torch.as_tensor(a) for name, a in out.items()}
