"""Plain float64 forms of graph attention, its distance buckets, the irreps layer norm and the
channel dropout.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).  Shares nothing with the CUDA library.

Attention, receiver by receiver and head by head: with head h owning the h-th part of every
block's channels (all components m),

    s[e, h] = scale <q[i], k[j]>_h + table[bucket[e], h],  p = softmax of s over the edges into i,
    y[i]_h = sum_e r[e, h] p[e, h] v[j]_h,                 lse[i, h] = log sum_e exp s[e, h].

Edges whose bucket or sender is out of range, and per head edges whose table entry is -inf, are
left out; a receiver without edges has y = 0 and lse = -inf.  Gradients are torch autograd VJPs.

Norm: per block, 0e blocks lose their mean over channels, every block is divided by the root of
its mean square over channels and components (+ eps) and scaled per channel; 0e blocks get a bias.

Dropout: value number n of Philox4x32-10 (Salmon, Moraes, Dror, Shaw, SC 2011), n = row * channels
+ channel (norm-free rows) or edge * heads + head (probabilities), kept when not below round(p 2^32).
"""
from __future__ import annotations

from typing import List, Optional

import numpy as np
import torch

from .irreps import Irreps

__all__ = ["head_columns", "attention", "attention_backward", "distance_buckets", "norm", "norm_backward",
           "philox_words", "keep_values", "dropout"]


def _t(a) -> Optional[torch.Tensor]:
    if a is None:
        return None
    if isinstance(a, torch.Tensor):
        return a.detach().to("cpu", torch.float64)
    return torch.as_tensor(np.asarray(a), dtype=torch.float64)


def head_columns(irreps: str, heads: int) -> List[np.ndarray]:
    """The columns of a row that each head owns."""
    ir = Irreps(irreps)
    cols: List[List[int]] = [[] for _ in range(heads)]
    for (mul, l, _), off in zip(ir.blocks, ir.offsets):
        d = 2 * l + 1
        for u in range(mul):
            cols[u * heads // mul].extend(range(off + u * d, off + (u + 1) * d))
    return [np.array(c) for c in cols]


def _attention_t(irreps_qk, irreps_v, heads, rowptr, src, q, k, v, bucket, table, n_buckets, scale, r):
    N, E = len(rowptr) - 1, len(src)
    src = np.asarray(src)
    live = (src >= 0) & (src < N)
    if bucket is not None:
        bucket = np.asarray(bucket)
        live &= (bucket >= 0) & (bucket < n_buckets)
    cq, cv = head_columns(irreps_qk, heads), head_columns(irreps_v, heads)
    y_rows, lse_rows = [], []
    for i in range(N):
        edges = [e for e in range(int(rowptr[i]), int(rowptr[i + 1])) if live[e]]
        y_row = torch.zeros(v.shape[1], dtype=torch.float64)
        lse_row = [torch.tensor(-float("inf"), dtype=torch.float64)] * heads
        for h in range(heads):
            mine = edges
            if table is not None:
                mine = [e for e in edges if float(table.detach()[bucket[e], h]) != -float("inf")]
            if not mine:
                continue
            j = src[mine]
            s = scale * (k[j][:, cq[h]] @ q[i][cq[h]])
            if table is not None:
                s = s + table[bucket[mine], h]
            top = s.detach().max()
            w = torch.exp(s - top)
            p = w / w.sum()
            if r is not None:
                p = p * r[mine, h]
            y_row = y_row.index_copy(0, torch.as_tensor(cv[h]), p @ v[j][:, cv[h]])
            lse_row[h] = top + torch.log(w.sum())
        y_rows.append(y_row)
        lse_rows.append(torch.stack(lse_row))
    if not N:
        return torch.zeros(0, v.shape[1], dtype=torch.float64), torch.zeros(0, heads, dtype=torch.float64)
    return torch.stack(y_rows), torch.stack(lse_rows)


def attention(irreps_qk, irreps_v, heads, rowptr, src, q, k, v, bucket=None, table=None, n_buckets=0, scale=1.0, r=None):
    """(y, lse) in float64; r [E, heads] are the dropout factors."""
    return _attention_t(irreps_qk, irreps_v, heads, rowptr, src, _t(q), _t(k), _t(v), bucket, _t(table), n_buckets,
                        scale, _t(r))


def attention_backward(irreps_qk, irreps_v, heads, rowptr, src, q, k, v, gy, bucket=None, table=None, n_buckets=0,
                       scale=1.0, r=None):
    """{"y", "lse", "gq", "gk", "gv", "gtable"} in float64."""
    q, k, v = (_t(a).clone().requires_grad_(True) for a in (q, k, v))
    table = None if table is None else _t(table).clone().requires_grad_(True)
    y, lse = _attention_t(irreps_qk, irreps_v, heads, rowptr, src, q, k, v, bucket, table, n_buckets, scale, _t(r))
    leaves = [q, k, v] + ([table] if table is not None else [])
    zero = sum((a * 0.0).nan_to_num(0.0).sum() for a in leaves)
    g = torch.autograd.grad((y * _t(gy)).sum() + zero, leaves)
    g = [torch.where(torch.isnan(a) & ~torch.isfinite(b), torch.zeros_like(a), a) for a, b in zip(g, leaves)]
    out = {"y": y.detach(), "lse": lse.detach(), "gq": g[0], "gk": g[1], "gv": g[2]}
    if table is not None:
        out["gtable"] = g[3]
    return out


def distance_buckets(vec, bounds, cutoff=None):
    """int32 [E]: number of bounds <= |vec|, -1 from the cutoff on and for NaN; compared as float64 squares."""
    v, b = np.asarray(vec, dtype=np.float64), np.asarray(bounds, dtype=np.float64)
    out = np.empty(len(v), dtype=np.int32)
    for e, (x, y, z) in enumerate(v):
        d2 = x * x + y * y + z * z
        n = sum(1 for t in b if t < 0 or d2 >= t * t)
        cut = np.inf if cutoff is None else float(np.float32(cutoff)) ** 2
        out[e] = n if d2 < cut else -1
    return out


def _norm_t(irreps, x, weight, bias, eps):
    ir = Irreps(irreps)
    rows, w0, b0 = [], 0, 0
    for (mul, l, parity), off in zip(ir.blocks, ir.offsets):
        d = 2 * l + 1
        b = x[:, off:off + mul * d].reshape(-1, mul, d)
        scalar = l == 0 and parity == 1
        if scalar:
            b = b - b.mean(dim=1, keepdim=True)
        n = b / torch.sqrt((b ** 2).mean(dim=(1, 2), keepdim=True) + eps)
        if weight is not None:
            n = n * weight[w0:w0 + mul].reshape(1, mul, 1)
        if scalar and bias is not None:
            n = n + bias[b0:b0 + mul].reshape(1, mul, 1)
        if scalar:
            b0 += mul
        w0 += mul
        rows.append(n.reshape(x.shape[0], mul * d))
    return torch.cat(rows, dim=1)


def norm(irreps, x, weight=None, bias=None, eps=1e-5):
    return _norm_t(irreps, _t(x), _t(weight), _t(bias), eps)


def norm_backward(irreps, x, gy, weight=None, bias=None, eps=1e-5):
    """{"gx", "gweight", "gbias"}; the weight and bias gradients exist whether or not they are given."""
    ir = Irreps(irreps)
    n_w = sum(mul for mul, _, _ in ir.blocks)
    n_b = sum(mul for mul, l, p in ir.blocks if l == 0 and p == 1)
    x = _t(x).clone().requires_grad_(True)
    w = (torch.ones(n_w, dtype=torch.float64) if weight is None else _t(weight).clone()).requires_grad_(True)
    b = (torch.zeros(n_b, dtype=torch.float64) if bias is None else _t(bias).clone()).requires_grad_(True)
    y = _norm_t(irreps, x, w, b, eps)
    gx, gw, gb = torch.autograd.grad((y * _t(gy)).sum() + 0.0 * b.sum(), (x, w, b))
    return {"gx": gx, "gweight": gw, "gbias": gb}


def philox_words(seed: int, offset: int, n: int) -> np.ndarray:
    """The first n 32-bit words: word n mod 4 of the block with counter (n div 4, offset) and key seed."""
    M0, M1, W0, W1, mask = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85, 0xFFFFFFFF
    out = []
    for block in range((n + 3) // 4):
        c = [block & mask, block >> 32, offset & mask, (offset >> 32) & mask]
        k0, k1 = seed & mask, (seed >> 32) & mask
        for _ in range(10):
            a, b = M0 * c[0], M1 * c[2]
            c = [(b >> 32) ^ c[1] ^ k0, b & mask, (a >> 32) ^ c[3] ^ k1, a & mask]
            k0, k1 = (k0 + W0) & mask, (k1 + W1) & mask
        out.extend(c)
    return np.array(out[:n], dtype=np.uint64)


def keep_values(seed: int, offset: int, n: int, p: float) -> np.ndarray:
    """n factors: 0 for a dropped value, 1 / (1 - p) for a kept one."""
    return np.where(philox_words(seed, offset, n) >= round(p * 2.0 ** 32), 1.0 / (1.0 - p), 0.0)


def dropout(irreps, x, p, seed, offset):
    ir = Irreps(irreps)
    x = _t(x)
    C = sum(mul for mul, _, _ in ir.blocks)
    r = torch.as_tensor(keep_values(seed, offset, x.shape[0] * C, p)).reshape(x.shape[0], C)
    widths = torch.tensor([2 * l + 1 for mul, l, _ in ir.blocks for _ in range(mul)])
    r = r.repeat_interleave(widths, dim=1)
    return torch.where(r > 0, x * r, torch.zeros_like(x))
