"""The forms of the attention kernels that sizes choose between: window lengths by the number of edges, windows of
one head group at a time, tables beside and behind the sender pass, and buckets four edges a thread."""
import numpy as np
import pytest
import torch

import attn_fast
from attn_util import assert_within, attn_bounds
from test_gpu_attn import OFFSET, SEED, SITE, check, dev, fast_buckets, problem, solve, tp  # noqa: F401

pytestmark = pytest.mark.gpu


def check_fast(pr, got):
    """test_gpu_attn.check for graphs that the loops of its oracle are too slow for."""
    d, E = pr["d"], int(pr["d"]["rowptr"][-1])
    r = attn_fast.keep_values(SEED, OFFSET + SITE, E * pr["heads"], pr["p"]).reshape(E, -1) if pr["p"] else None
    more = dict(bucket=d["bucket"], table=d["table"], n_buckets=pr["n_buckets"], scale=pr["scale"], r=r)
    x = [d[name] for name in ("q", "k", "v", "gy")]
    want = attn_fast.attention_backward(pr["qk"], pr["v"], pr["heads"], d["rowptr"], d["src"], *x, **more)
    bound = attn_bounds(pr["qk"], pr["v"], pr["heads"], d["rowptr"], d["src"], *x, want["lse"].numpy(), **more)
    for name in want:
        # the bounds grow with the terms of a sum; the library's stated 1e-4 of the largest value holds beside them
        if name != "lse":
            bound[name] = np.minimum(bound[name], 1e-4 * float(want[name].abs().max()))
        assert_within(got[name], want[name], bound[name], name)


def graph(rng, n, edges, long_rows):
    """`edges` edges over n rows: rows 3, 10, 17, ... of the given lengths, the rest spread evenly; every fifth
    edge comes from node 1, so the sender order has a long row too."""
    counts = np.zeros(n, int)
    at = 3 + 7 * np.arange(len(long_rows))
    counts[at] = long_rows
    others = np.setdiff1d(np.arange(n), at)
    left = edges - counts.sum()
    counts[others] = left // len(others)
    counts[others[:left % len(others)]] += 1
    src = rng.integers(0, n, edges).astype(np.int32)
    src[::5] = 1
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), src


@pytest.mark.parametrize("edges", [127, 128, 129, 319, 320, 321])
def test_where_windows_begin(tp, edges):
    rowptr = np.array([0, 0, edges, edges, edges], np.int32)
    pr = problem(50, "12x0e+4x1o", "12x0e+4x1o", 4, 4, 0, p=0.1, graph=(rowptr, np.full(edges, 2, np.int32)))
    check(pr, solve(tp, pr))


@pytest.mark.parametrize("n", [1500, 300])
@pytest.mark.parametrize("edges", [37887, 37888, 94719, 94720, 94721])
def test_windows_that_grow_with_the_edges(tp, edges, n):
    """64 to 160 edges a window, with rows around twice that, in graphs of one and of several warps a row."""
    rows = [127, 128, 129, 191, 192, 193, 255, 256, 257, 319, 320, 321, 383, 384, 385, 3001, 0, 1]
    pr = problem(51, "4x0e", "4x0e+2x1o", 2, n, 0, p=0.1, graph=graph(np.random.default_rng(edges), n, edges, rows))
    for transposed in (True, False):
        check_fast(pr, solve(tp, pr, transposed))


@pytest.mark.parametrize("edges", [378879, 378880, 500001])
def test_windows_beyond_160_edges(tp, edges):
    rows = [319, 320, 321, 383, 384, 385, 447, 448, 449, 5001, 20000]
    pr = problem(52, "2x0e", "1x1o+1x0e", 1, 4001, 0, graph=graph(np.random.default_rng(1), 4001, edges, rows))
    check_fast(pr, solve(tp, pr))


@pytest.mark.parametrize("qk,v,heads", [("128x0e+128x1o+128x2e", "128x0e+128x1o+128x2e", 8), ("24x0e", "120x0e+24x1o", 6),
                                        ("21x0e+21x1o", "21x0e+21x1o+21x2e+21x3o", 7), ("600x0e", "8x0e", 2)])
def test_windows_of_one_head_group_at_a_time(tp, qk, v, heads):
    """Enough rows for one warp each, heads that fill more than one warp, and long rows."""
    n = 1301
    pr = problem(53, qk, v, heads, n, 0, p=0.2, graph=graph(np.random.default_rng(2), n, 9001, [1000, 129, 128, 127, 700]))
    d = pr["d"]
    d["bucket"][d["rowptr"][3]:d["rowptr"][3] + 200] = -1      # windows that are masked as a whole
    d["table"][3, heads - 1] = -np.inf
    check_fast(pr, solve(tp, pr))


@pytest.mark.parametrize("buckets,heads", [(1024, 8), (1025, 8), (4096, 2), (4096, 8), (1024, 32), (4096, 1), (256, 32), (129, 16)])
@pytest.mark.parametrize("n", [1301, 40])
def test_large_tables(tp, buckets, heads, n):
    """Up to 32,768 entries, on both sides of the 8,192 that a sender pass's CTA keeps a copy of."""
    irreps = f"{heads}x0e+{heads}x1o"
    pr = problem(54, irreps, irreps, heads, n, 0, n_buckets=buckets, p=0.1,
                 graph=graph(np.random.default_rng(3), n, 20011, [900, 300]))
    d = pr["d"]
    d["bucket"][:6000] = buckets - 1                           # one entry of thousands of edges
    d["table"][5 % buckets, 0] = -np.inf
    whole = solve(tp, pr)
    check_fast(pr, whole)
    alone = solve(tp, pr, need_gq=False, need_gk=False, need_gv=False)
    want, size = whole["gtable"].double(), whole["gtable"].double().abs().max()
    assert float((alone["gtable"].double() - want).abs().max()) <= 1e-4 * float(size)


def test_a_large_table_of_a_whole_cta_a_head(tp):
    pr = problem(55, "301x0e", "301x3o", 1, 30, 0, n_buckets=4096, graph=graph(np.random.default_rng(4), 30, 1501, [400, 300]))
    check_fast(pr, solve(tp, pr))


@pytest.mark.parametrize("E", [151551, 151552, 151553, 151554, 151555, 1300001])
@pytest.mark.parametrize("n_bounds", [0, 1, 31, 32, 255, 1023])
def test_buckets_four_edges_a_thread(tp, E, n_bounds):
    rng = np.random.default_rng(E)
    vec = (rng.standard_normal((E, 3)) * 2).astype(np.float32)
    bounds = np.sort(rng.uniform(0.1, 6.0, n_bounds)).astype(np.float32)
    special = [[0, 0, 0], [np.nan, 1, 1], [np.inf, 0, 0], [0, -np.inf, 1], [5, 0, 0], [0, 3, 4], [1e-30, 0, 0], [3e38, 3e38, 3e38]]
    vec[:len(special)] = special
    for i, b in enumerate(bounds):
        vec[-1 - i] = np.roll([b, 0, 0], i)                    # exactly on a bound, and one step below it
        if i % 2:
            vec[-1 - i] = np.nextafter(vec[-1 - i], np.float32(0))
    for cutoff in (None, 5.0):
        want = fast_buckets(vec, bounds, cutoff)
        # aligned, and vec and bucket one to three floats off a 16-byte boundary: one edge a thread
        for at, to in ((0, 0), (1, 0), (0, 1), (2, 3)):
            flat = torch.zeros(3 * E + at, device="cuda")
            flat[at:] = dev(vec).flatten()
            out = torch.full((E + to + 1,), 77, dtype=torch.int32, device="cuda")
            got = tp.tp_distance_buckets(flat[at:].view(E, 3), dev(bounds), cutoff, bucket=out[to:to + E])
            np.testing.assert_array_equal(got.cpu().numpy(), want)
            assert bool((out[:to] == 77).all()) and int(out[to + E]) == 77
