"""Graphs, inputs and derived error bounds of the graph-attention tests.

The bounds follow the formulas term by term with u = 2^-24 (fp32, round to nearest: at most half
a step): a sum of n products of which each is off by at most n u of the sum of the absolute
values; exp and log off by 2^-21 relative / 2^-22 absolute (the error of the hardware's exp2 and
log2, two units in the last place, and of the argument's scaling, which adds |argument| u)."""
from __future__ import annotations

import numpy as np

from oracle.attn import head_columns

U = 2.0 ** -24


def random_graph(rng, n, mean_degree, spare=0, empty=0.1):
    """Receiver CSR with random degrees (some zero) and `spare` edges behind the last row."""
    counts = rng.poisson(mean_degree, n) * (rng.random(n) >= empty)
    rowptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    src = rng.integers(0, max(n, 1), rowptr[-1] + spare).astype(np.int32)
    return rowptr, src


def attn_bounds(irreps_qk, irreps_v, heads, rowptr, src, q, k, v, gy, lse, bucket=None, table=None, n_buckets=0,
                scale=1.0, r=None):
    """Largest allowed |error| of y, lse, gq, gk, gv, gtable, element by element."""
    N = len(rowptr) - 1
    rowptr, src = np.asarray(rowptr), np.asarray(src)
    E = int(rowptr[-1])
    dst = np.repeat(np.arange(N), np.diff(rowptr))
    src = src[:E]
    live = (src >= 0) & (src < N)
    if bucket is not None:
        bucket = np.asarray(bucket)[:E]
        live &= (bucket >= 0) & (bucket < n_buckets)
    e = np.nonzero(live)[0]
    i, j = dst[e], src[e]
    deg = np.bincount(i, minlength=N).max(initial=0)
    out_deg = np.bincount(j, minlength=N).max(initial=0)
    f = lambda a: np.nan_to_num(np.asarray(a, dtype=np.float64), nan=0.0, posinf=0.0, neginf=0.0)
    q, k, v, gy, L = f(q), f(k), f(v), f(gy), f(lse)
    zero = lambda a: np.zeros_like(a)
    out = {"y": zero(v), "lse": zero(L), "gq": zero(q), "gk": zero(k), "gv": zero(v),
           "gtable": np.zeros((max(n_buckets, 1), heads))}
    for h, (cq, cv) in enumerate(zip(head_columns(irreps_qk, heads), head_columns(irreps_v, heads))):
        qk = scale * (q[i][:, cq] * k[j][:, cq])
        a, s = np.abs(qk).sum(1), qk.sum(1)
        bias, keep = np.zeros(len(e)), np.ones(len(e), bool)
        if table is not None:
            raw = np.asarray(table, dtype=np.float64)[bucket[e], h]
            keep = raw != -np.inf
            bias = np.where(keep, raw, 0.0)
        s = s + bias
        p = np.where(keep, np.exp(np.minimum(s - L[i, h], 0.0)), 0.0)
        ds = U * ((len(cq) + 3) * a + 2 * np.abs(bias) + np.abs(s))
        ds = np.where(keep, ds, 0.0)
        ds_row = np.zeros(N)
        np.maximum.at(ds_row, i, ds)
        dl = ds_row + (deg + 4) * U + 2.0 ** -22 + 2 * U * np.abs(L[:, h])
        out["lse"][:, h] = dl
        near = np.minimum(np.abs(s - L[i, h]), 90.0)           # beyond it p is 0 either way
        rho = float(np.max(np.where(p > 0, ds + dl[i] + 4 * near * U, 0.0), initial=0.0)) + 2.0 ** -21
        rr = np.ones(len(e)) if r is None else np.asarray(r)[e, h]
        c_y = 2 * rho + (deg + 8) * U
        ybar = np.zeros((N, len(cv)))
        np.add.at(ybar, i, (p * rr)[:, None] * np.abs(v[j][:, cv]))
        out["y"][:, cv] = c_y * ybar
        t = rr * (np.abs(gy[i][:, cv]) * np.abs(v[j][:, cv])).sum(1) + (np.abs(gy[i][:, cv]) * ybar[i]).sum(1)
        c_d = 2 * rho + c_y + (len(cv) + 8) * U
        g = np.zeros((N, len(cq)))
        np.add.at(g, i, (scale * p * t)[:, None] * np.abs(k[j][:, cq]))
        out["gq"][:, cq] = (c_d + (deg + 4) * U) * g
        g = np.zeros((N, len(cq)))
        np.add.at(g, j, (scale * p * t)[:, None] * np.abs(q[i][:, cq]))
        out["gk"][:, cq] = (c_d + (out_deg + 4) * U) * g
        g = np.zeros((N, len(cv)))
        np.add.at(g, j, (rr * p)[:, None] * np.abs(gy[i][:, cv]))
        out["gv"][:, cv] = (2 * rho + (out_deg + 4) * U) * g
        if table is not None:
            g = np.zeros(max(n_buckets, 1))
            np.add.at(g, bucket[e], p * t)
            out["gtable"][:, h] = (c_d + (E + 8) * U) * g
    tiny = 1e-30                                               # results below 2^-126 are flushed to zero
    return {name: b + tiny for name, b in out.items()}


def assert_within(got, want, bound, name):
    g = np.asarray(got.detach().double().cpu())
    w = np.asarray(want.detach().double())
    assert g.shape == w.shape, (name, g.shape, w.shape)
    same = (g == w) | (np.isnan(g) & np.isnan(w))
    with np.errstate(invalid="ignore"):
        off = np.abs(g - w)
    bad = ~same & ~(off <= bound)
    if bad.any():
        at = np.unravel_index(np.argmax(np.where(bad, np.nan_to_num(off / bound, nan=np.inf), 0)), g.shape)
        raise AssertionError(f"{name}: {int(bad.sum())} of {g.size} off, worst at {at}: {g[at]!r} against {w[at]!r}, "
                             f"allowed {np.broadcast_to(bound, g.shape)[at]:.3e}")
