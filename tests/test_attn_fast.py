"""The fast forms of tests/attn_fast.py against the loops of oracle/attn.py."""
import numpy as np
import pytest
import torch

import attn_fast
from attn_util import random_graph
from oracle import attn as oa
from oracle.irreps import Irreps


@pytest.mark.parametrize("n,p", [(1, 0.3), (4, 0.2), (1003, 0.1), (20000, 0.999)])
def test_keep_values(n, p):
    np.testing.assert_array_equal(attn_fast.keep_values(-5 % 2 ** 64, 7 << 33, n, p), oa.keep_values(-5 % 2 ** 64, 7 << 33, n, p))


@pytest.mark.parametrize("buckets", [0, 4])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_attention(buckets, p):
    rng = np.random.default_rng(buckets)
    qk, v, heads, n = "8x0e+4x1o", "4x0e+8x1o+4x2e", 4, 23
    rowptr, src = random_graph(rng, n, 6)
    src[::11] = -1
    src[5::13] = n
    E, f = len(src), lambda *s: rng.standard_normal(s).astype(np.float32)
    more = dict(scale=0.3)
    if buckets:
        table = f(buckets, heads)
        table[1, 2] = -np.inf
        more.update(bucket=rng.integers(-1, buckets + 1, E), table=table, n_buckets=buckets)
    if p:
        more["r"] = oa.keep_values(1, 2, E * heads, p).reshape(E, heads)
    x = [f(n, Irreps(a).dim) for a in (qk, qk, v, v)]
    want = oa.attention_backward(qk, v, heads, rowptr, src, *x, **more)
    got = attn_fast.attention_backward(qk, v, heads, rowptr, src, *x, **more)
    assert set(got) == set(want)
    for name in want:
        # float64 sums of some tens of terms of size one
        assert torch.equal(torch.isinf(got[name]), torch.isinf(want[name]))
        assert float(torch.nan_to_num(got[name] - want[name], nan=0.0).abs().max()) < 1e-12, name
