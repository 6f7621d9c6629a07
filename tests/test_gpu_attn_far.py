"""Backward passes of attention rows whose logits all lie far from zero: a constant in the table, or the lowest
float as a mask on every edge of a row.  The softmax of such a row is that of its unshifted logits, which
lse, rounded to 32 bits, no longer tells."""
import math

import numpy as np
import pytest
import torch

import attn_fast
from attn_util import assert_within, attn_bounds
from oracle.attn import head_columns
from oracle.irreps import Irreps
from test_gpu_attn import OFFSET, SEED, SITE, solve, tp  # noqa: F401

pytestmark = pytest.mark.gpu

# four warps a receiver and one, windows of both, 16- and 4-byte rows, a whole CTA a head
FORMS = [("8x0e+4x1o", "8x0e+4x1o", 4, 14), ("64x0e", "32x0e+32x1o+32x2e+32x3o", 8, 14), ("21x0e+21x1o", "21x0e+21x1o+21x2e", 3, 14),
         ("301x0e", "301x3o", 1, 14), ("1100x0e", "8x0e", 1, 14), ("8x0e+4x1o", "8x0e+4x1o", 4, 1300), ("128x0e", "128x0e+128x1o", 2, 1300)]


def graph(rng, n):
    counts = rng.poisson(6, n)
    counts[:9] = [3, 900, 0, 130, 700, 40, 1, 257, 64]
    rowptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return rowptr, rng.integers(0, n, rowptr[-1]).astype(np.int32)


def integers(qk, v, heads, n, seed, p):
    """q and k of small whole numbers and a power of two as scale: every logit and its sum with the shift below
    is exact in 32 bits, in any order of summation."""
    rng = np.random.default_rng(seed)
    rowptr, src = graph(rng, n)
    width = Irreps(qk).dim // heads
    scale = 2.0 ** -math.ceil(math.log2(2 * math.sqrt(width)))
    whole = lambda: rng.integers(-2, 3, (n, Irreps(qk).dim)).astype(np.float32)
    f = lambda: rng.standard_normal((n, Irreps(v).dim)).astype(np.float32)
    d = dict(rowptr=rowptr, src=src, q=whole(), k=whole(), v=f(), gy=f())
    # odd rows use bucket 0, even rows bucket 1; bucket 2 masks one head, -1 the edge
    row = np.repeat(np.arange(n), np.diff(rowptr))
    d["bucket"] = np.where(row % 2 == 1, 0, 1).astype(np.int32)
    d["bucket"][rng.random(len(src)) < 0.1] = 2
    d["bucket"][rng.random(len(src)) < 0.1] = -1
    d["table"] = np.zeros((3, heads), np.float32)
    d["table"][2, heads - 1] = -np.inf
    return dict(qk=qk, v=v, heads=heads, n_buckets=3, p=p, scale=scale, d=d)


def reference(pr, table):
    d = pr["d"]
    E = len(d["src"])
    r = attn_fast.keep_values(SEED, OFFSET + SITE, E * pr["heads"], pr["p"]).reshape(E, -1) if pr["p"] else None
    more = dict(bucket=d["bucket"], table=table, n_buckets=3, scale=pr["scale"], r=r)
    x = [d[name] for name in ("q", "k", "v", "gy")]
    want = attn_fast.attention_backward(pr["qk"], pr["v"], pr["heads"], d["rowptr"], d["src"], *x, **more)
    return want, lambda q, k: attn_bounds(pr["qk"], pr["v"], pr["heads"], d["rowptr"], d["src"], q, k, d["v"], d["gy"],
                                          want["lse"].numpy(), **more)


def records(pr):
    """The most maxima that a row's logits pass on the way to their largest, in edge order."""
    d, most = pr["d"], 0
    for h, c in enumerate(head_columns(pr["qk"], pr["heads"])):
        for i in range(len(d["rowptr"]) - 1):
            e = slice(d["rowptr"][i], d["rowptr"][i + 1])
            s = (d["k"][d["src"][e]][:, c] @ d["q"][i, c])[d["bucket"][e] >= 0]
            if len(s):
                most = max(most, len(np.unique(np.maximum.accumulate(s))))
    return most


@pytest.mark.parametrize("qk,v,heads,n", FORMS)
@pytest.mark.parametrize("shift", [2.0 ** 11, -2.0 ** 11, 2.0 ** 16, -2.0 ** 16])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_a_constant_in_the_table_changes_no_gradient(tp, qk, v, heads, n, shift, p):
    pr = integers(qk, v, heads, n, 31, p)
    pr["d"]["table"][0, ::2] = shift                           # bucket 2 joins rows of bucket 0: keep those apart
    pr["d"]["table"][2, ::2] += np.float32(shift)
    near = np.repeat(np.arange(n), np.diff(pr["d"]["rowptr"])) % 2 == 0
    pr["d"]["bucket"][near & (pr["d"]["bucket"] == 2)] = 1
    want, bounds = reference(pr, np.where(np.isinf(pr["d"]["table"]), -np.inf, 0.0).astype(np.float32))
    bound = bounds(pr["d"]["q"], pr["d"]["k"])
    got = solve(tp, pr)
    # the bounds assume a sum of exponentials below one maximum; each maximum passed on the way multiplies it by
    # one more exponential, off by 2^-21, against 2^-20 that every bound holds at least
    slack = 1 + (records(pr) + 2) / 2
    for name in ("y", "gq", "gk", "gv", "gtable"):
        assert_within(got[name], want[name], slack * bound[name], name)


@pytest.mark.parametrize("qk,v,heads,n", FORMS)
@pytest.mark.parametrize("mask", [np.finfo(np.float32).min, -1e30])
def test_rows_masked_by_the_lowest_float(tp, qk, v, heads, n, mask):
    """q.k vanishes beside the mask, so every probability is one over the row's live edges."""
    pr = integers(qk, v, heads, n, 32, 0.25)
    d = pr["d"]
    d["table"][0] = mask
    d["bucket"][d["bucket"] == 2] = -1
    want, bounds = reference(pr, d["table"])
    # the bounds of equal logits, in the rows that have them: q = 0 there for all but gk, which grows with q alone
    q0, table = d["q"].copy(), d["table"].copy()
    q0[1::2] = 0
    table[0] = 0
    _, flat = reference(dict(pr, d=dict(d, q=q0)), table)
    bound = flat(q0, d["k"])
    bound["gk"] = flat(d["q"], 0 * d["k"])["gk"] + flat(q0, d["k"])["gk"]
    got = solve(tp, pr)
    slack = 1 + (records(pr) + 2) / 2
    for name in ("y", "gq", "gk", "gv", "gtable"):
        assert_within(got[name], want[name], slack * bound[name], name)
