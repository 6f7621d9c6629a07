"""Graph attention and the distance buckets on the GPU against the float64 forms, within error
bounds derived from the formulas (tests/attn_util.py), at the sizes, masks and layouts where
they can go wrong."""
import math

import numpy as np
import pytest
import torch

from attn_util import assert_within, attn_bounds, random_graph
from oracle import attn as oa
from oracle.irreps import Irreps

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tp():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from equivariant_tensor_product_b200 import build
    build.build()
    import equivariant_tensor_product_b200 as tp
    return tp


def dev(a, dtype=None):
    t = torch.as_tensor(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


SEED, OFFSET, SITE = 0x1234567890ABCDEF, (5 << 32) + 7, 3


def problem(seed, qk, v, heads, n, mean_degree, n_buckets=5, p=0.0, spare=0, graph=None):
    rng = np.random.default_rng(seed)
    rowptr, src = random_graph(rng, n, mean_degree, spare) if graph is None else graph
    E = len(src)
    f = lambda *s: rng.standard_normal(s).astype(np.float32)
    d = dict(rowptr=rowptr, src=src, q=f(n, Irreps(qk).dim), k=f(n, Irreps(qk).dim), v=f(n, Irreps(v).dim),
             gy=f(n, Irreps(v).dim), bucket=None, table=None)
    if n_buckets:
        d["bucket"] = rng.integers(-1, n_buckets, E).astype(np.int32)
        d["table"] = f(n_buckets, heads)
    return dict(qk=qk, v=v, heads=heads, n_buckets=n_buckets, p=p, scale=float(np.float32(math.sqrt(heads / Irreps(qk).dim))), d=d)


def solve(tp, pr, transposed=True, **kw):
    """The library's results for a problem."""
    d = pr["d"]
    attn = tp.Attention(pr["qk"], pr["v"], pr["heads"], pr["n_buckets"])
    g = {k: None if a is None else dev(a) for k, a in d.items()}
    rng = torch.tensor([SEED, OFFSET], dtype=torch.int64, device="cuda") if pr["p"] else None
    more = dict(bucket=g["bucket"], table=g["table"], scale=pr["scale"], p=pr["p"], rng=rng, site=SITE)
    y, lse = tp.tp_attn_fwd(attn, g["rowptr"], g["src"], g["q"], g["k"], g["v"], **more)
    colptr = perm = None
    if transposed:
        colptr, perm = tp.tp_csr_transpose(g["rowptr"], g["src"], len(d["rowptr"]) - 1)
    gq, gk, gv, gt = tp.tp_attn_bwd(attn, g["rowptr"], g["src"], g["q"], g["k"], g["v"], y, lse, g["gy"], colptr=colptr,
                                    perm=perm, **more, **kw)
    return {"y": y, "lse": lse, "gq": gq, "gk": gk, "gv": gv, "gtable": gt}


def check(pr, got, names=("y", "lse", "gq", "gk", "gv", "gtable")):
    d = pr["d"]
    E = int(d["rowptr"][-1])
    r = None
    if pr["p"]:
        r = oa.keep_values(SEED, OFFSET + SITE, E * pr["heads"], pr["p"]).reshape(E, pr["heads"])
    args = dict(bucket=None if d["bucket"] is None else d["bucket"][:E], table=d["table"], n_buckets=pr["n_buckets"],
                scale=pr["scale"], r=r)
    want = oa.attention_backward(pr["qk"], pr["v"], pr["heads"], d["rowptr"], d["src"][:E], d["q"], d["k"], d["v"], d["gy"], **args)
    bound = attn_bounds(pr["qk"], pr["v"], pr["heads"], d["rowptr"], d["src"], d["q"], d["k"], d["v"], d["gy"], want["lse"].numpy(),
                        **args)
    for name in names:
        if name in want:
            assert_within(got[name], want[name], bound[name], name)
    return want


# heads with one to many chunks a lane, 16-byte and 4-byte rows, one warp and a whole CTA per head
SHAPES = [
    ("4x0e+4x1o", "4x0e+4x1o", 2), ("1x0e", "1x0e", 1), ("1x1o", "1x3o", 1), ("5x0e+5x1o", "5x2e", 5), ("21x0e+21x1o", "21x0e+21x1o+21x2e", 3),
    ("8x0e", "32x0e+32x1o+32x2e", 4), ("32x0e+32x1o+32x2e", "32x0e+32x1o+32x2e", 4), ("64x0e", "64x0e+64x1o+64x2e+64x3o", 8),
    ("64x0e+64x1o+64x2e+64x3o", "64x0e", 32), ("32x0o", "32x1e+32x0o", 32), ("12x0e+24x0e", "12x1o+12x1e", 12),
    ("16x0e+16x2e", "160x0e+32x1o", 1), ("33x0e+33x1o+33x2e", "33x0e+33x1o", 1), ("128x0e+128x1o", "128x0e+128x1o+128x2e", 1),
    ("100x0e+100x3o", "118x0e+118x2e", 1), ("600x0e", "300x1o+64x0e", 2), ("4x0e", "512x3o", 1), ("301x0e", "301x3o", 1),
    ("128x0e+128x0o+128x1o+128x1e+128x2e+128x3o", "8x0e", 1), ("32x0e+32x1o+32x2e+32x3o", "32x0e+32x1o+32x2e+32x3o", 8),
    ("128x0e+128x1o", "512x0e", 32), ("256x0e", "256x1o+128x0e", 16),
]


@pytest.mark.parametrize("qk,v,heads", SHAPES)
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_shapes(tp, qk, v, heads, p):
    pr = problem(1, qk, v, heads, n=17, mean_degree=9, p=p, spare=3)
    check(pr, solve(tp, pr))


@pytest.mark.parametrize("n,degree", [(1, 0), (1, 1), (1, 40), (2, 1), (3, 33), (40, 0.3), (64, 31), (64, 64), (300, 3), (5, 300)])
@pytest.mark.parametrize("heads", [1, 4])
def test_lengths(tp, n, degree, heads):
    rng = np.random.default_rng(n)
    counts = np.full(n, degree, int) if degree >= 1 else rng.integers(0, 2, n)
    rowptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    pr = problem(2, "8x0e+4x1o", "8x0e+4x1o", heads, n, degree, p=0.2,
                 graph=(rowptr, rng.integers(0, n, rowptr[-1]).astype(np.int32)))
    for transposed in (True, False):
        check(pr, solve(tp, pr, transposed))


@pytest.mark.parametrize("buckets", [0, 1, 200])
def test_without_and_with_many_buckets(tp, buckets):
    pr = problem(3, "8x0e", "8x0e+8x1o", 2, n=50, mean_degree=12, n_buckets=buckets)
    got = solve(tp, pr)
    assert (got["gtable"] is None) == (buckets == 0)
    check(pr, got)
    if buckets:                                                # a mask alone: buckets without a table
        pr["d"]["table"] = None
        check(pr, solve(tp, pr))


def test_receivers_and_senders_of_very_many_edges(tp):
    """One node hears and tells all others: rows of thousands of edges next to rows of a few."""
    n = 3001
    rng = np.random.default_rng(4)
    dst = np.concatenate([rng.integers(0, n - 1, 6000), np.full(n - 1, n - 1), np.arange(n - 1), np.full(700, 5)])
    src = np.concatenate([rng.integers(0, n - 1, 6000), np.arange(n - 1), np.full(n - 1, n - 1), np.full(700, 9)])
    order = np.argsort(dst, kind="stable")
    rowptr = np.concatenate([[0], np.cumsum(np.bincount(dst, minlength=n))]).astype(np.int32)
    for qk, v, heads, p in (("8x0e+4x1o", "8x0e+4x1o", 4, 0.25), ("3x0e", "3x1o", 3, 0.0)):
        pr = problem(5, qk, v, heads, n, 0, p=p, graph=(rowptr, src[order].astype(np.int32)))
        check(pr, solve(tp, pr))


@pytest.mark.parametrize("edges", [255, 256, 257, 511, 512, 513, 640, 1025, 5000])
def test_one_receiver_and_its_edges(tp, edges):
    """Few rows and a long axis: all edges into node 1, all from node 2, and rows without edges around."""
    rowptr = np.array([0, 0, edges, edges, edges], np.int32)
    pr = problem(6, "12x0e+4x1o", "12x0e+4x1o", 4, 4, 0, p=0.1, graph=(rowptr, np.full(edges, 2, np.int32)))
    check(pr, solve(tp, pr))


@pytest.mark.parametrize("qk,v,heads", [("64x0e+32x1o+32x2e", "64x0e+32x1o+32x3o", 8), ("301x0e", "301x3o", 1), ("2x0e+2x1o", "130x0e", 2), ("1x0e", "129x0e", 1)])
def test_long_rows_of_many_floats(tp, qk, v, heads):
    """Rows of 63 to 193 edges, around the shortest window and twice it, whose joins are cut by the floats of the
    row; one of them in windows that are masked as a whole."""
    counts = np.array([3, 127, 128, 0, 129, 130, 63, 64, 65, 193, 1, 160, 2, 191])
    n, rng = len(counts), np.random.default_rng(8)
    rowptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    src = rng.integers(0, n, rowptr[-1]).astype(np.int32)
    src[rng.random(len(src)) < 0.3] = 7                        # a sender of some 400 edges
    pr = problem(9, qk, v, heads, n, 0, p=0.2, graph=(rowptr, src))
    d = pr["d"]
    d["bucket"][rowptr[9]:rowptr[9] + 140] = -1
    d["bucket"][rowptr[5]:rowptr[6]] = -1                      # and a long row that hears nobody
    got = solve(tp, pr)
    assert bool((got["lse"][5] == -math.inf).all()) and bool((got["y"][5] == 0).all()) and bool((got["gq"][5] == 0).all())
    check(pr, got)


def test_masks_that_leave_a_row_nothing(tp):
    pr = problem(7, "8x0e+4x1o", "8x0e+4x1o", 4, n=30, mean_degree=6, spare=5)
    d = pr["d"]
    at = lambda i: slice(int(d["rowptr"][i]), int(d["rowptr"][i + 1]))
    d["bucket"][at(3)] = -1
    d["bucket"][at(4)] = 99                                    # beyond the table
    d["src"][at(5)] = -1
    d["src"][at(6)] = 30
    d["bucket"][at(7)] = 2
    d["table"][2, 1] = -np.inf                                 # one head of one bucket
    got = solve(tp, pr)
    want = check(pr, got)
    for i in (3, 4, 5, 6):
        assert bool((got["y"][i] == 0).all()) and bool((got["lse"][i] == -math.inf).all()) and bool((got["gq"][i] == 0).all())
    assert float(want["lse"][7, 1]) == -math.inf or at(7).start == at(7).stop
    d["table"][:] = -np.inf
    got = solve(tp, pr)
    for name in ("y", "gq", "gk", "gv", "gtable"):
        assert bool((got[name] == 0).all()), name


def test_lowest_value_in_the_table_is_a_number(tp):
    """A row whose every logit is near the lowest float is an ordinary softmax of equal logits."""
    pr = problem(8, "8x0e", "8x0e+4x1o", 2, n=20, mean_degree=6)
    pr["d"]["table"][1] = np.finfo(np.float32).min
    pr["d"]["table"][3] = -1e30
    lowest = np.nonzero(np.diff(pr["d"]["rowptr"]))[0][0]
    pr["d"]["bucket"][pr["d"]["rowptr"][lowest]:pr["d"]["rowptr"][lowest + 1]] = 1
    got = solve(tp, pr)
    d = pr["d"]
    j = d["src"][d["rowptr"][lowest]:d["rowptr"][lowest + 1]]
    mean = d["v"][j].astype(np.float64).mean(0)
    # q.k vanishes beside 3.4e38, so every probability is 1 / degree
    assert_within(got["y"][lowest], torch.as_tensor(mean), 2.0 ** -18 * np.abs(d["v"][j]).max(0) + 1e-30, "y")
    pr["d"]["table"][1] = -1e30
    check(pr, solve(tp, pr), names=("y", "gv"))


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_what_a_masked_row_holds_reaches_nothing(tp, value):
    """Node 0 only sends along masked edges, node 1 receives nothing: their rows may hold anything."""
    pr = problem(9, "8x0e+4x1o", "8x0e+4x1o", 4, n=25, mean_degree=7, p=0.2)
    d = pr["d"]
    d["table"][4] = -np.inf
    from_zero = d["src"] == 0
    d["bucket"][from_zero] = np.where(np.arange(from_zero.sum()) % 2, -1, 4)
    lo, hi = d["rowptr"][1], d["rowptr"][2]
    d["bucket"][lo:hi] = np.where(np.arange(hi - lo) % 2, -1, 4)
    clean = solve(tp, pr)
    for name in ("k", "v"):
        d[name][0] = value
    for name in ("q", "gy"):
        d[name][1] = value
    got = solve(tp, pr)
    keep = np.arange(25)
    for name in ("y", "lse", "gq", "gk", "gv", "gtable"):
        assert torch.equal(got[name], clean[name]), name
    check(pr, got)


def test_a_nan_or_infinity_in_play_shows(tp):
    pr = problem(10, "8x0e", "8x0e", 2, n=20, mean_degree=6, n_buckets=0)
    pr["d"]["k"][3, 0] = math.nan
    got = solve(tp, pr)
    d = pr["d"]
    hears = [i for i in range(20) if 3 in d["src"][d["rowptr"][i]:d["rowptr"][i + 1]]]
    assert hears
    for i in range(20):
        assert bool(torch.isnan(got["y"][i, :4]).all()) == (i in hears)        # head 0 alone
        assert not bool(torch.isnan(got["y"][i, 4:]).any())


@pytest.mark.parametrize("shift", [0, 1])
def test_column_slices_in_and_out(tp, shift):
    """q, k, v and their gradients as slices of one array, 16-byte aligned and not; what lies between stays."""
    pr = problem(11, "16x0e+16x1o", "16x0e+16x1o+16x2e", 4, n=40, mean_degree=8, p=0.1, spare=4)
    d = pr["d"]
    plain = solve(tp, pr)
    dq, dv, n = 64, 144, 40
    width = 2 * dq + dv + 12
    cols = {"q": slice(shift, shift + dq), "k": slice(dq + 4, 2 * dq + 4), "v": slice(2 * dq + 8 - shift, 2 * dq + dv + 8 - shift)}
    big, gbig = torch.full((n, width), 7.0, device="cuda"), torch.full((n, width), 7.0, device="cuda")
    for name, c in cols.items():
        big[:, c] = dev(d[name])
    attn = tp.Attention(pr["qk"], pr["v"], pr["heads"], pr["n_buckets"])
    rng = torch.tensor([SEED, OFFSET], dtype=torch.int64, device="cuda")
    more = dict(bucket=dev(d["bucket"]), table=dev(d["table"]), scale=pr["scale"], p=pr["p"], rng=rng, site=SITE)
    rows = (dev(d["rowptr"]), dev(d["src"]), big[:, cols["q"]], big[:, cols["k"]], big[:, cols["v"]])
    y, lse = tp.tp_attn_fwd(attn, *rows, **more)
    gt = tp.tp_attn_bwd(attn, *rows, y, lse, dev(d["gy"]), gq=gbig[:, cols["q"]], gk=gbig[:, cols["k"]], gv=gbig[:, cols["v"]],
                        **more)[3]
    check(pr, {"y": y, "lse": lse, "gq": gbig[:, cols["q"]], "gk": gbig[:, cols["k"]], "gv": gbig[:, cols["v"]], "gtable": gt})
    if shift == 0:
        assert torch.equal(y, plain["y"]) and torch.equal(gbig[:, cols["v"]], plain["gv"])
    used = torch.zeros(width, dtype=torch.bool)
    for c in cols.values():
        used[c] = True
    assert bool((gbig[:, ~used] == 7.0).all())
    with pytest.raises(ValueError, match="contiguous rows"):
        tp.tp_attn_fwd(attn, rows[0], rows[1], big[:, :2 * dq:2], *rows[3:], **more)
    with pytest.raises(ValueError, match="contiguous rows"):
        tp.tp_attn_fwd(attn, rows[0], rows[1], big[:1, cols["q"]].expand(n, dq), *rows[3:], **more)


def test_row_offsets_beyond_32_bits(tp):
    """Rows so far apart that the last ones start beyond 2^31 floats (and 2^32 bytes) of the array."""
    n, ld = 300, 8_000_000
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of device memory")
    pr = problem(12, "4x0e+4x1o", "4x0e+4x1o", 2, n=n, mean_degree=5)
    d = pr["d"]
    big = torch.empty(n * ld, device="cuda")
    view = lambda at: big.as_strided((n, 16), (ld, 1), at)
    for at, name in ((0, "q"), (16, "k"), (32, "v")):
        view(at).copy_(dev(d[name]))
    attn = tp.Attention(pr["qk"], pr["v"], pr["heads"], pr["n_buckets"])
    more = dict(bucket=dev(d["bucket"]), table=dev(d["table"]), scale=pr["scale"])
    rows = (dev(d["rowptr"]), dev(d["src"]), view(0), view(16), view(32))
    y, lse = tp.tp_attn_fwd(attn, *rows, **more)
    gq, gk, gv, gt = tp.tp_attn_bwd(attn, *rows, y, lse, dev(d["gy"]), gq=view(64), gk=view(80), gv=view(96), **more)
    check(pr, {"y": y, "lse": lse, "gq": gq, "gk": gk, "gv": gv, "gtable": gt})


def test_each_gradient_alone_and_none(tp):
    pr = problem(13, "8x0e", "8x0e+8x1o", 2, n=40, mean_degree=9)
    whole = solve(tp, pr)
    for name in ("gq", "gk", "gv", "gtable"):
        want = {f"need_{n}": n == name for n in ("gq", "gk", "gv", "gtable")}
        got = solve(tp, pr, **want)
        assert torch.equal(got[name], whole[name])
        assert all(got[n] is None for n in ("gq", "gk", "gv", "gtable") if n != name)
    attn = tp.Attention("8x0e", "8x0e+8x1o", 2, 5)
    d = {k: dev(a) for k, a in pr["d"].items()}
    y, lse = tp.tp_attn_fwd(attn, d["rowptr"], d["src"], d["q"], d["k"], d["v"], bucket=d["bucket"], table=d["table"],
                            scale=pr["scale"], need_lse=False)
    assert lse is None and torch.equal(y, whole["y"])


def test_results_repeat_bit_for_bit(tp):
    pr = problem(14, "32x0e+32x1o+32x2e", "32x0e+32x1o+32x2e", 4, n=500, mean_degree=40, p=0.1)
    a, b = solve(tp, pr), solve(tp, pr, transposed=False)
    for name in a:
        assert torch.equal(a[name], b[name]), name


def test_spare_edges_and_poisoned_buffers(tp):
    """A list of fixed capacity: what stands behind the last row's edges is never used, and every output and
    workspace byte may hold NaNs before the call."""
    pr = problem(15, "8x0e", "8x0e", 2, n=30, mean_degree=6, spare=50, p=0.2)
    d = pr["d"]
    want = solve(tp, pr)
    d["src"][d["rowptr"][-1]:] = np.arange(50) % 30            # valid senders and buckets, still no row's edges
    d["bucket"][d["rowptr"][-1]:] = 1
    attn = tp.Attention("8x0e", "8x0e", 2, 5)
    g = {k: dev(a) for k, a in d.items()}
    nan = lambda *s: torch.full(s, math.nan, device="cuda")
    E = len(d["src"])
    ws = torch.full(((tp.tp_attn_workspace_size(attn, 30, E, tp.TP_OP_BWD) + 3) // 4,), math.nan, device="cuda").view(torch.uint8)
    more = dict(bucket=g["bucket"], table=g["table"], scale=pr["scale"], p=0.2,
                rng=torch.tensor([SEED, OFFSET], dtype=torch.int64, device="cuda"), site=SITE)
    rows = (g["rowptr"], g["src"], g["q"], g["k"], g["v"])
    y, lse = tp.tp_attn_fwd(attn, *rows, y=nan(30, 8), lse=nan(30, 2), ws=ws, **more)
    got = tp.tp_attn_bwd(attn, *rows, y, lse, g["gy"], gq=nan(30, 8), gk=nan(30, 8), gv=nan(30, 8), gtable=nan(5, 2), ws=ws, **more)
    got = dict(zip(("y", "lse", "gq", "gk", "gv", "gtable"), (y, lse) + got))
    check(pr, got)
    for name in ("y", "lse", "gq"):                            # gk, gv: a sender's sums may be cut elsewhere
        assert torch.equal(got[name], want[name]), name
    with pytest.raises(ValueError, match="workspace"):
        tp.tp_attn_bwd(attn, *rows, y, lse, g["gy"], ws=ws[:256], **more)


@pytest.mark.parametrize("before", [1, 300, 700])
def test_spare_edges_before_the_first_row(tp, before):
    """rowptr[0] > 0: the edges before it belong to no row, next to receivers and senders of very many edges."""
    rng = np.random.default_rng(20)
    counts = rng.poisson(6, 40)
    counts[0], counts[7], counts[39] = 900, 1300, 700
    rowptr = np.concatenate([[0], np.cumsum(counts)])
    src = rng.integers(0, 40, rowptr[-1])
    src[rng.random(len(src)) < 0.4] = 11
    pr = problem(20, "8x0e+4x1o", "8x0e+4x1o", 4, 40, 0, graph=(rowptr.astype(np.int32), src.astype(np.int32)))
    want = check(pr, solve(tp, pr))
    d = pr["d"]
    d["rowptr"] = (d["rowptr"] + before).astype(np.int32)
    for name, values in (("src", rng.integers(0, 40, before)), ("bucket", rng.integers(0, 5, before))):
        d[name] = np.concatenate([values, d[name]]).astype(np.int32)
    for transposed in (True, False):
        got = solve(tp, pr, transposed)
        bound = attn_bounds(pr["qk"], pr["v"], 4, d["rowptr"] - before, d["src"][before:], d["q"], d["k"], d["v"], d["gy"],
                            want["lse"].numpy(), bucket=d["bucket"][before:], table=d["table"], n_buckets=5, scale=pr["scale"])
        for name in want:
            assert_within(got[name], want[name], bound[name], name)


def test_graphs_without_edges_or_nodes(tp):
    attn = tp.Attention("8x0e", "8x0e", 2, 5)
    z = lambda *s: torch.zeros(*s, device="cuda")
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
    for n in (0, 7):
        x = torch.ones(n, 8, device="cuda")
        more = dict(bucket=i32(0), table=torch.ones(5, 2, device="cuda"))
        y, lse = tp.tp_attn_fwd(attn, i32(n + 1), i32(0), x, x, x, **more)
        assert y.shape == (n, 8) and bool((y == 0).all()) and bool((lse == -math.inf).all())
        out = tp.tp_attn_bwd(attn, i32(n + 1), i32(0), x, x, x, y, lse, x, gtable=torch.ones(5, 2, device="cuda"), **more)
        assert all(bool((t == 0).all()) for t in out) and out[3].shape == (5, 2)


def test_captured_calls_draw_anew_and_do_not_share(tp):
    """Two graphs with workspaces of their own, replayed in turn and at once on two streams; the offset moves
    inside the captured step."""
    prs = [problem(16 + i, "8x0e+4x1o", "8x0e+4x1o", 4, n=60, mean_degree=9, p=0.4) for i in (0, 1)]
    graphs, alive = [], []
    for pr in prs:
        attn = tp.Attention(pr["qk"], pr["v"], pr["heads"], pr["n_buckets"])
        g = {k: dev(a) for k, a in pr["d"].items()}
        colptr, perm = tp.tp_csr_transpose(g["rowptr"], g["src"], 60)
        rng = torch.tensor([SEED, OFFSET - 1], dtype=torch.int64, device="cuda")
        more = dict(bucket=g["bucket"], table=g["table"], scale=pr["scale"], p=pr["p"], rng=rng, site=SITE)
        rows = (g["rowptr"], g["src"], g["q"], g["k"], g["v"])

        def step(rows=rows, g=g, more=more, attn=attn, colptr=colptr, perm=perm, rng=rng):
            rng[1] += 1
            y, lse = tp.tp_attn_fwd(attn, *rows, **more)
            return (y, lse) + tp.tp_attn_bwd(attn, *rows, y, lse, g["gy"], colptr=colptr, perm=perm, **more)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, out, rng))
        alive.append(step)                                     # a graph reads its inputs where they were
    for pr, (graph, out, rng) in zip(prs, graphs):
        graph.replay()
    torch.cuda.synchronize()
    first = []
    for pr, (graph, out, rng) in zip(prs, graphs):
        check(pr, dict(zip(("y", "lse", "gq", "gk", "gv", "gtable"), out)))
        first.append([t.clone() for t in out])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for (graph, out, rng) in graphs:
        rng[1] = OFFSET - 1
    torch.cuda.synchronize()
    for (graph, out, rng), s in zip(graphs, streams):
        with torch.cuda.stream(s):
            graph.replay()
    torch.cuda.synchronize()
    for (graph, out, rng), f in zip(graphs, first):
        assert all(torch.equal(a, b) for a, b in zip(out, f))
    graphs[0][0].replay()                                      # the next offset: another mask
    torch.cuda.synchronize()
    assert not torch.equal(graphs[0][1][0], first[0][0])


def test_on_another_stream(tp):
    pr = problem(18, "8x0e", "8x0e+8x1o", 2, n=400, mean_degree=20)
    want = solve(tp, pr)
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        s.wait_stream(torch.cuda.current_stream())
        got = solve_on(tp, pr, stream)
        torch.cuda.current_stream().wait_stream(s)
        for name in want:
            assert torch.equal(got[name], want[name]), name


def solve_on(tp, pr, stream):
    d = {k: dev(a) for k, a in pr["d"].items()}
    torch.cuda.synchronize()
    attn = tp.Attention(pr["qk"], pr["v"], pr["heads"], pr["n_buckets"])
    more = dict(bucket=d["bucket"], table=d["table"], scale=pr["scale"], stream=stream)
    rows = (d["rowptr"], d["src"], d["q"], d["k"], d["v"])
    y, lse = tp.tp_attn_fwd(attn, *rows, **more)
    out = tp.tp_attn_bwd(attn, *rows, y, lse, d["gy"], **more)
    torch.cuda.synchronize()
    return dict(zip(("y", "lse", "gq", "gk", "gv", "gtable"), (y, lse) + out))


@pytest.mark.parametrize("E", [1, 2, 3, 4, 5, 255, 1027, 70001])
@pytest.mark.parametrize("n_bounds", [0, 1, 31, 1023])
def test_distance_buckets(tp, E, n_bounds):
    rng = np.random.default_rng(E + n_bounds)
    vec = (rng.standard_normal((E, 3)) * 2).astype(np.float32)
    bounds = np.sort(rng.uniform(0.1, 6.0, n_bounds)).astype(np.float32)
    special = [[0, 0, 0], [math.nan, 1, 1], [math.inf, 0, 0], [0, -math.inf, 1], [5, 0, 0], [0, 3, 4], [1e-30, 0, 0],
               [3e38, 3e38, 3e38], [1e-45, 0, 0]]
    for i, s in enumerate(special[:max(0, E - 1)]):
        vec[i] = s
    for i, b in enumerate(bounds[:max(0, E - len(special))]):
        vec[-1 - i] = np.roll([b, 0, 0], i)                    # exactly on a bound, and one step below it
        if i % 2:
            vec[-1 - i] = np.nextafter(vec[-1 - i], np.float32(0))
    for cutoff in (None, 5.0, 0.0, math.inf):
        got = tp.tp_distance_buckets(dev(vec), dev(bounds), cutoff).cpu().numpy()
        np.testing.assert_array_equal(got, fast_buckets(vec, bounds, cutoff))
    if E * max(1, n_bounds) <= 300000:
        np.testing.assert_array_equal(fast_buckets(vec, bounds, 5.0), oa.distance_buckets(vec, bounds, 5.0))


def fast_buckets(vec, bounds, cutoff):
    v, b = vec.astype(np.float64), bounds.astype(np.float64)
    with np.errstate(invalid="ignore"):
        d2 = v[:, 0] * v[:, 0] + v[:, 1] * v[:, 1] + v[:, 2] * v[:, 2]
        n = np.searchsorted(b * b, d2, side="right")
        return np.where(d2 < (np.inf if cutoff is None else np.float64(np.float32(cutoff)) ** 2), n, -1)


def test_buckets_of_an_unaligned_slice(tp):
    rng = np.random.default_rng(0)
    flat = dev(rng.standard_normal(3 * 500 + 3).astype(np.float32))
    bounds = dev(np.linspace(0.2, 3, 9).astype(np.float32))
    for at in (0, 1, 2, 3):
        vec = flat[at:at + 1500].view(500, 3)
        got = tp.tp_distance_buckets(vec, bounds, 2.5)
        np.testing.assert_array_equal(got.cpu().numpy(), fast_buckets(vec.cpu().numpy(), bounds.cpu().numpy(), 2.5))
    out = torch.full((502,), 77, dtype=torch.int32, device="cuda")
    tp.tp_distance_buckets(flat[:1500].view(500, 3), bounds, 2.5, bucket=out[1:501])
    assert int(out[0]) == 77 and int(out[501]) == 77


def test_outputs_in_place_of_inputs_are_refused(tp):
    """Other rows' sums still read q, k, v and gy while a row's outputs are written."""
    pr = problem(40, "8x0e", "8x0e", 2, n=20, mean_degree=5)
    g = {k: dev(a) for k, a in pr["d"].items()}
    attn = tp.Attention("8x0e", "8x0e", 2, 5)
    rows, more = (g["rowptr"], g["src"], g["q"], g["k"], g["v"]), dict(bucket=g["bucket"], table=g["table"])
    for name in ("q", "k", "v"):
        with pytest.raises(ValueError, match="share memory"):
            tp.tp_attn_fwd(attn, *rows, y=g[name], **more)
    y, lse = tp.tp_attn_fwd(attn, *rows, y=torch.empty(20, 8, device="cuda"), **more)
    own = torch.empty(20, 8, device="cuda")
    for given in (dict(gq=g["q"]), dict(gk=g["k"]), dict(gv=g["gy"]), dict(gv=y), dict(gtable=g["table"]), dict(gq=own, gk=own)):
        with pytest.raises(ValueError, match="share memory"):
            tp.tp_attn_bwd(attn, *rows, y, lse, g["gy"], **given, **more)
    tp.tp_attn_bwd(attn, *rows, y, lse, g["gy"], gq=own, **more)


def test_a_sender_order_first_made_on_another_stream(tp):
    """A backward call on one stream while the order that it shares is still being built on another."""
    pr = problem(41, "8x0e+4x1o", "8x0e+4x1o", 4, n=400, mean_degree=20)
    want = solve(tp, pr)
    d = {k: dev(a) for k, a in pr["d"].items()}
    attn, graph = tp.Attention(pr["qk"], pr["v"], pr["heads"], pr["n_buckets"]), tp.autograd.Graph(d["rowptr"], d["src"])
    q, k, v = (d[name].requires_grad_(True) for name in ("q", "k", "v"))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            y = tp.tp_attn(attn, graph, q, k, v, d["bucket"], d["table"], pr["scale"])
            if i == 0:
                torch.cuda._sleep(50_000_000)                  # some 25 ms before the order is built
            got.append(torch.autograd.grad(y, (q, k, v), d["gy"]))
    torch.cuda.synchronize()
    for grads in got:
        for g, name in zip(grads, ("gq", "gk", "gv")):
            assert torch.equal(g, want[name]), name
