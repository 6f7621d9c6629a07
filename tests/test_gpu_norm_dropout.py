"""The irreps layer norm and the channel dropout on the GPU against the float64 forms, and a whole
attention layer (norm, linear, buckets, attention, linear, dropout) differentiated through
autograd."""
import math

import numpy as np
import pytest
import torch

from attn_util import U, assert_within, random_graph
from oracle import attn as oa
from oracle import block as ob
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


def dev(a):
    return torch.as_tensor(np.ascontiguousarray(a)).cuda()


def norm_bounds(irreps, x, w, b, gy, eps):
    """Allowed errors of y, gx, gweight, gbias.  A block of L floats: the mean is off by (L + 2) u mean|x|, so
    c = x - mean by a = that + u |c|; the mean square by (L + 4) u of itself and twice |mean c| a, which
    vanishes but for rounding; rho by half that and 2^-21 (the hardware's reciprocal root); n = c rho by
    rho a + |n| (k u + 2^-21), and so on through the formulas."""
    ir = Irreps(irreps)
    N, dim = x.shape
    f = lambda a: np.asarray(a, np.float64)
    x, gy = f(x), f(gy)
    out = {"y": np.zeros((N, dim)), "gx": np.zeros((N, dim)), "gweight": [], "gbias": []}
    w0 = b0 = 0
    for (mul, l, parity), off in zip(ir.blocks, ir.offsets):
        d, L = 2 * l + 1, mul * (2 * l + 1)
        scalar = l == 0 and parity == 1
        xb, gb = x[:, off:off + L], gy[:, off:off + L]
        mu = xb.mean(1, keepdims=True) if scalar else np.zeros((N, 1))
        c = xb - mu
        a = ((L + 2) * U * np.abs(xb).mean(1, keepdims=True) if scalar else 0.0) + U * np.abs(c)
        ms = (c * c).mean(1, keepdims=True) + eps
        rho = 1 / np.sqrt(ms)
        rel = 0.5 * ((L + 4) * U + 2 * (a * np.abs(c)).mean(1, keepdims=True) / ms + U) + 2.0 ** -21
        n = c * rho
        dn = rho * a + np.abs(n) * (rel + 2 * U)
        wb = np.repeat(np.ones(mul) if w is None else f(w)[w0:w0 + mul], d)
        bb = np.repeat(f(b)[b0:b0 + mul], d) if scalar and b is not None else np.zeros(L)
        y = n * wb + bb
        out["y"][:, off:off + L] = np.abs(wb) * dn + 2 * U * (np.abs(n * wb) + np.abs(y)) + 1e-30
        g = gb * wb
        s1 = (L + 3) * U * np.abs(g).mean(1, keepdims=True)
        s2 = (np.abs(g) * (dn + (L + 4) * U * np.abs(n))).mean(1, keepdims=True)
        m2 = np.abs((g * n).mean(1, keepdims=True))
        size = np.abs(g) + np.abs(g).mean(1, keepdims=True) + np.abs(n) * m2
        out["gx"][:, off:off + L] = rho * ((rel + 6 * U) * size + s1 + s2 * np.abs(n) + m2 * dn) + 1e-30
        t = (np.abs(gb) * (dn + (N * d + 4) * U * np.abs(n))).reshape(N, mul, d).sum((0, 2))
        out["gweight"].append(t + 1e-30)
        if scalar:
            out["gbias"].append((N + 2) * U * np.abs(gb).sum(0) + 1e-30)
            b0 += mul
        w0 += mul
    out["gweight"] = np.concatenate(out["gweight"])
    out["gbias"] = np.concatenate(out["gbias"]) if out["gbias"] else np.zeros(0)
    return out


NORMS = [("1x0e", 1), ("1x0e", 70), ("7x0e", 33), ("64x0e", 1), ("64x0e", 1000), ("16x0e", 517), ("4x0e+4x1o", 24), ("32x0e+32x1o+32x2e", 300),
         ("21x0e+21x1o+21x2e+21x3o", 65), ("3x1o", 9), ("5x0o+3x0e+2x0e", 40), ("128x0e+128x1o+128x2e", 700), ("64x0e+64x1o+64x2e+64x3o", 130),
         ("160x0e+160x0o+160x1o+160x1e+160x2e+160x3o", 37), ("8192x0e", 5), ("1001x0e+999x3o", 3), ("+".join(["4x1o", "4x0e"] * 8), 50),
         ("4x0e+4x1o+4x2e", 5000), ("8x0e", 20001)]


@pytest.mark.parametrize("irreps,rows", NORMS)
@pytest.mark.parametrize("affine", [True, False])
def test_norm(tp, irreps, rows, affine):
    rng = np.random.default_rng(rows)
    norm = tp.Norm(irreps)
    f = lambda *s: rng.standard_normal(s).astype(np.float32)
    x, gy = f(rows, norm.dim) * 3 + 1, f(rows, norm.dim)
    w, b = (f(norm.n_weights), f(norm.n_bias)) if affine else (None, None)
    on = lambda a: None if a is None else dev(a)
    y = tp.tp_norm_fwd(norm, dev(x), on(w), on(b))
    gx, gw, gb = tp.tp_norm_bwd(norm, dev(x), dev(gy), on(w))
    want = oa.norm_backward(irreps, x, gy, w, b)
    want["y"] = oa.norm(irreps, x, w, b)
    bound = norm_bounds(irreps, x, w, b, gy, 1e-5)
    for got, name in ((y, "y"), (gx, "gx"), (gw, "gweight"), (gb, "gbias")):
        assert_within(got, want[name], bound[name], name)


def test_norm_of_special_rows(tp):
    """Zero rows, equal channels, huge and tiny rows, and a row with a NaN beside clean ones."""
    irreps, rng = "16x0e+8x1o", np.random.default_rng(0)
    x = rng.standard_normal((8, 40)).astype(np.float32)
    x[0] = 0
    x[1, :16] = 3.0
    x[2] *= 1e15
    x[3] *= 1e-15
    x[4, 0] = math.nan
    x[5, 20] = math.inf
    y = tp.tp_norm_fwd(tp.Norm(irreps), dev(x)).cpu().numpy()
    assert (y[0] == 0).all() and (y[1, :16] == 0).all()
    assert np.isnan(y[4, :16]).all() and np.isfinite(y[4, 16:]).all()
    assert np.isfinite(y[5, :16]).all() and np.isnan(y[5, 20])
    clean = [0, 1, 2, 3, 6, 7]
    bound = norm_bounds(irreps, x[clean], None, None, x[clean], 1e-5)["y"]
    assert_within(torch.as_tensor(y[clean]), oa.norm(irreps, x[clean]), bound, "y")


@pytest.mark.parametrize("irreps", ["32x0e+32x1o", "7x0e+5x1o"])
def test_norm_in_place_parts_and_layouts(tp, irreps):
    norm, rng = tp.Norm(irreps), np.random.default_rng(1)
    f = lambda *s: dev(rng.standard_normal(s).astype(np.float32))
    x, gy, w, b = f(77, norm.dim), f(77, norm.dim), f(norm.n_weights), f(norm.n_bias)
    y = tp.tp_norm_fwd(norm, x, w, b)
    gx, gw, gb = tp.tp_norm_bwd(norm, x, gy, w)
    again = x.clone()
    assert tp.tp_norm_fwd(norm, again, w, b, y=again) is again and torch.equal(again, y)
    own = gy.clone()
    tp.tp_norm_bwd(norm, x, own, w, gx=own)
    assert torch.equal(own, gx)
    for name, want in (("gx", gx), ("gweight", gw), ("gbias", gb)):
        got = tp.tp_norm_bwd(norm, x, gy, w, **{f"need_{n}": n == name for n in ("gx", "gweight", "gbias")})
        assert sum(t is not None for t in got) == 1
        assert torch.equal(next(t for t in got if t is not None), want)
    buf, gbuf = torch.full((77 * norm.dim + 2,), 5.0, device="cuda"), torch.full((77 * norm.dim + 2,), 5.0, device="cuda")
    odd = buf[1:-1].view(77, norm.dim)                        # rows that start 4 bytes off
    odd.copy_(x)
    bound = norm_bounds(irreps, x.cpu().numpy(), w.cpu().numpy(), b.cpu().numpy(), gy.cpu().numpy(), 1e-5)
    assert_within(tp.tp_norm_fwd(norm, odd, w, b, y=gbuf[1:-1].view(77, norm.dim)), oa.norm(irreps, x, w, b), bound["y"], "y")
    assert float(gbuf[0]) == 5.0 and float(gbuf[-1]) == 5.0
    r = tp.tp_norm_bwd(norm, odd, gy, w)
    want = oa.norm_backward(irreps, x, gy, w, b)
    for t, name in zip(r, ("gx", "gweight", "gbias")):
        assert_within(t, want[name], bound[name], name)


@pytest.mark.parametrize("irreps,rows,start", [("2x0e", 1, 0), ("6x0e+2x1o", 45, 0), ("18x0o+18x1o+18x1e+18x2e", 391, 0), ("78x0o+78x1o+78x2e+78x3o", 130, 0),
                                               ("1150x0e+6x0e", 40, 0), ("382x1o", 33, 0), ("30x0e+30x3o", 2003, 0), ("64x0e+32x1o", 130, 2),
                                               ("1152x0e", 21, 2), ("8x0e", 1000, 2)])
def test_norm_of_eight_byte_rows(tp, irreps, rows, start):
    """Blocks of an even number of floats that is no multiple of four, and rows that start 8 bytes off."""
    norm, rng = tp.Norm(irreps), np.random.default_rng(rows)
    f = lambda *s: rng.standard_normal(s).astype(np.float32)
    x, gy, w, b = f(rows, norm.dim) * 3 + 1, f(rows, norm.dim), f(norm.n_weights), f(norm.n_bias)

    def laid(a):
        buf = torch.full((rows * norm.dim + start,), 5.0, device="cuda")
        buf[start:] = torch.as_tensor(a).cuda().flatten()
        return buf[start:].view(rows, norm.dim)

    y = tp.tp_norm_fwd(norm, laid(x), dev(w), dev(b), y=laid(gy))
    gx, gw, gb = tp.tp_norm_bwd(norm, laid(x), laid(gy), dev(w), gx=laid(x))
    want = oa.norm_backward(irreps, x, gy, w, b)
    want["y"] = oa.norm(irreps, x, w, b)
    bound = norm_bounds(irreps, x, w, b, gy, 1e-5)
    for got, name in ((y, "y"), (gx, "gx"), (gw, "gweight"), (gb, "gbias")):
        assert_within(got, want[name], bound[name], name)


def test_norm_of_no_rows_and_repeats(tp):
    norm = tp.Norm("8x0e+8x1o")
    x = torch.zeros(0, norm.dim, device="cuda")
    assert tp.tp_norm_fwd(norm, x).shape == (0, norm.dim)
    gx, gw, gb = tp.tp_norm_bwd(norm, x, x)
    assert gx.shape == (0, norm.dim) and bool((gw == 0).all()) and bool((gb == 0).all())
    g = torch.Generator("cuda").manual_seed(0)
    x, gy = (torch.randn(30011, norm.dim, generator=g, device="cuda") for _ in range(2))
    a, b = tp.tp_norm_bwd(norm, x, gy), tp.tp_norm_bwd(norm, x, gy)
    assert all(torch.equal(s, t) for s, t in zip(a, b))


@pytest.mark.parametrize("irreps,rows", [("1x0e", 1), ("1x0e", 5), ("3x1o", 7), ("4x0e+4x1o", 100), ("7x0e+5x1o+3x2e", 61),
                                         ("32x0e+32x1o+32x2e", 50), ("5000x0e", 2), ("1100x3o", 2), ("128x0e+128x1o+128x2e", 33)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.999])
def test_dropout(tp, irreps, rows, p):
    drop, rng = tp.Dropout(irreps), np.random.default_rng(rows)
    x = rng.standard_normal((rows, drop.dim)).astype(np.float32)
    seed, offset, site = -7, 1 << 40, 5
    r = torch.tensor([seed, offset], dtype=torch.int64, device="cuda")
    y = tp.tp_dropout_fwd(drop, dev(x), p, r, site)
    want = oa.dropout(irreps, x, p, seed % (1 << 64), offset + site)
    # one rounding of 1/(1-p) and one of the product
    assert_within(y, want, 2 * U * np.abs(want.numpy()) * (1 + 2 * U), "y")
    assert torch.equal(y == 0, (want == 0).cuda() | (dev(x) == 0))
    assert torch.equal(tp.tp_dropout_bwd(drop, dev(x), p, r, site), y)
    own = dev(x)
    assert tp.tp_dropout_fwd(drop, own, p, r, site, y=own) is own and torch.equal(own, y)
    buf = torch.full((rows * drop.dim + 2,), 5.0, device="cuda")
    tp.tp_dropout_fwd(drop, dev(x), p, r, site, y=buf[1:-1].view(rows, drop.dim))
    assert torch.equal(buf[1:-1].view(rows, drop.dim), y) and float(buf[0]) == 5.0 and float(buf[-1]) == 5.0


def test_dropped_values_may_hold_anything(tp):
    drop = tp.Dropout("64x0e")
    r = torch.tensor([1, 2], dtype=torch.int64, device="cuda")
    y = tp.tp_dropout_fwd(drop, torch.full((100, 64), math.nan, device="cuda"), 0.5, r)
    gone = ~torch.isnan(y)
    assert 0.4 < float(gone.float().mean()) < 0.6 and bool((y[gone] == 0).all())
    assert tp.tp_dropout_fwd(drop, torch.zeros(0, 64, device="cuda"), 0.5, r).shape == (0, 64)


IR, MID, K, HEADS = "16x0e+8x1o", "16x0e+8x1o+16x0e+8x1o+16x0e+8x1o", 6, 4


def _layer(tp, P, x, graph, vec, rng, p):
    """A pre-norm attention layer: x + dropout(linear(attention(linear(norm(x)))))."""
    bucket = tp.tp_distance_buckets(vec, P["bounds"], 2.5)
    h = tp.tp_norm(P["norm"], x, P["weight"], P["bias"])
    qkv = tp.tp_linear(P["lin_in"], h, P["W_in"])
    a = tp.tp_attn(P["attn"], graph, qkv[:, :40], qkv[:, 40:80], qkv[:, 80:], bucket, P["table"], p=p, rng=rng, site=1)
    return x + tp.tp_dropout(P["drop"], tp.tp_linear(P["lin_out"], a, P["W_out"]), p, rng, site=2)


def _oracle_layer(P, x, rowptr, src, vec, p, seed, offset):
    leaves = {k: P[k].detach().double().cpu().requires_grad_(True) for k in ("weight", "bias", "W_in", "W_out", "table")}
    x = x.detach().double().cpu().requires_grad_(True)
    h = oa._norm_t(IR, x, leaves["weight"], leaves["bias"], 1e-5)
    qkv = ob._linear_t(IR, MID, h, leaves["W_in"], None)
    E, C = len(src), 24
    r = torch.as_tensor(oa.keep_values(seed, offset + 1, E * HEADS, p)).reshape(E, HEADS) if p else None
    bucket = oa.distance_buckets(vec, P["bounds"].cpu().numpy(), 2.5)
    y, _ = oa._attention_t(IR, IR, HEADS, rowptr, src, qkv[:, :40], qkv[:, 40:80], qkv[:, 80:], bucket, leaves["table"], K,
                           math.sqrt(HEADS / 40), r)
    out = ob._linear_t(IR, IR, y, leaves["W_out"], None)
    if p:
        keep = torch.as_tensor(oa.keep_values(seed, offset + 2, x.shape[0] * C, p)).reshape(-1, C)
        out = out * keep.repeat_interleave(torch.tensor([1] * 16 + [3] * 8), dim=1)
    return x + out, x, leaves


def _make_layer(tp, seed=0, n=40):
    rng = np.random.default_rng(seed)
    rowptr, src = random_graph(rng, n, 8)
    f = lambda *s: torch.as_tensor(rng.standard_normal(s).astype(np.float32)).cuda()
    P = dict(norm=tp.Norm(IR), lin_in=tp.Linear(IR, MID), lin_out=tp.Linear(IR, IR), attn=tp.Attention(IR, IR, HEADS, K),
             drop=tp.Dropout(IR), bounds=dev(np.linspace(0.5, 2.2, K - 1).astype(np.float32)))
    P.update(weight=1 + 0.1 * f(P["norm"].n_weights), bias=0.1 * f(P["norm"].n_bias), W_in=f(P["lin_in"].n_weights) / 4,
             W_out=f(P["lin_out"].n_weights) / 4, table=f(K, HEADS))
    vec = rng.standard_normal((len(src), 3)).astype(np.float32)
    return P, rowptr, src, vec, f(n, 40), f(n, 40)


@pytest.mark.parametrize("p", [0.0, 0.2])
def test_a_whole_layer_through_autograd(tp, p):
    P, rowptr, src, vec, x, gy = _make_layer(tp)
    names = ("weight", "bias", "W_in", "W_out", "table")
    for k in names:
        P[k].requires_grad_(True)
    x.requires_grad_(True)
    graph = tp.autograd.Graph(dev(rowptr), dev(src))
    rng = torch.tensor([3, 4], dtype=torch.int64, device="cuda")
    y = _layer(tp, P, x, graph, dev(vec), rng, p)
    got = torch.autograd.grad(y, [x] + [P[k] for k in names], gy)
    want_y, want_x, leaves = _oracle_layer(P, x, rowptr, src, vec, p, 3, 4)
    want = torch.autograd.grad(want_y, [want_x] + [leaves[k] for k in names], gy.double().cpu())
    # the library's stated fp32 tolerance, per tensor
    for g, w, name in zip((y,) + got, (want_y,) + want, ("y", "x") + names):
        err, scale = float((g.detach().double().cpu() - w.detach()).abs().max()), float(w.detach().abs().max())
        assert err <= 1e-4 * scale, (name, err, scale)
    # and against differences along a random direction, in the library's own forward
    step = torch.randn(x.shape, generator=torch.Generator().manual_seed(1)).cuda()
    with torch.no_grad():
        eps = 2.0 ** -7
        hi, lo = (_oracle_layer(P, x + s * eps * step, rowptr, src, vec, p, 3, 4)[0].detach() for s in (1, -1))
        num = float(((hi - lo) * gy.double().cpu()).sum() / (2 * eps))
    ana = float((got[0].double() * step.double()).sum())
    # central differences are off by eps^2 / 6 times a third derivative: of the order of the gradient's own size
    assert abs(num - ana) <= 40 * eps ** 2 * float(got[0].double().norm() * step.double().norm()) / math.sqrt(x.numel())


def test_layer_refuses_what_it_cannot_differentiate(tp):
    P, rowptr, src, vec, x, gy = _make_layer(tp)
    x.requires_grad_(True)
    graph = tp.autograd.Graph(dev(rowptr), dev(src))
    rng = torch.tensor([3, 4], dtype=torch.int64, device="cuda")
    y = _layer(tp, P, x, graph, dev(vec), rng, 0.2)
    (gx,) = torch.autograd.grad(y, x, gy, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(gx.sum(), x)                       # norm and attention are first order
    y = _layer(tp, P, x, graph, dev(vec), rng, 0.2)
    rng[1] += 1                                                # the mask of the forward call is gone
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(y, x, gy)
    # dropout is linear: differentiable twice
    drop = tp.Dropout(IR)
    v = torch.randn_like(x).requires_grad_(True)
    z = tp.tp_dropout(drop, x * v, 0.3, rng)
    (g,) = torch.autograd.grad((z ** 2).sum(), x, create_graph=True)
    (h,) = torch.autograd.grad(g.sum(), v)
    r = tp.tp_dropout_fwd(drop, torch.ones_like(x), 0.3, rng)
    want = 4 * r * r * x * v
    assert float((h - want).detach().abs().max()) <= 1e-5 * float(want.detach().abs().max())


def test_a_captured_layer(tp):
    """Forward and backward of the layer in one graph; replays with new inputs equal eager calls."""
    P, rowptr, src, vec, x, gy = _make_layer(tp)
    names = ("weight", "bias", "W_in", "W_out", "table")
    leaves = [x] + [P[k] for k in names]
    graph = tp.autograd.Graph(dev(rowptr), dev(src))
    graph.transpose()
    rng, vec = torch.tensor([3, 4], dtype=torch.int64, device="cuda"), dev(vec)
    for t in leaves:
        t.requires_grad_(True)

    def step():
        y = _layer(tp, P, x, graph, vec, rng, 0.2)
        return (y.detach(),) + torch.autograd.grad(y, leaves, gy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        out = step()
    with torch.no_grad():
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(2)))
        rng[1] = 9
    cg.replay()
    torch.cuda.synchronize()
    eager = step()
    assert all(torch.equal(a, b) for a, b in zip(out, eager))


def test_a_layer_captured_before_its_sender_order_exists(tp):
    """The captured backward builds the order itself and leaves the graph object without it."""
    P, rowptr, src, vec, x, gy = _make_layer(tp, seed=3)
    graph = tp.autograd.Graph(dev(rowptr), dev(src))
    q = torch.randn(40, 40, generator=torch.Generator().manual_seed(4)).cuda().requires_grad_(True)
    bucket = tp.tp_distance_buckets(dev(vec), P["bounds"], 2.5)
    step = lambda: torch.autograd.grad(tp.tp_attn(P["attn"], graph, q, q, q, bucket, P["table"]), q, gy)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.no_grad():
            tp.tp_attn(P["attn"], graph, q, q, q, bucket, P["table"])
    torch.cuda.current_stream().wait_stream(side)
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        out = step()
    assert graph._colptr is None
    eager = step()                                             # before the first replay
    cg.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager)


def test_calls_on_another_stream_than_the_current_one(tp):
    norm, drop = tp.Norm("32x0e+32x1o"), tp.Dropout("32x0e+32x1o")
    g = torch.Generator("cuda").manual_seed(0)
    x, gy = (torch.randn(3000, norm.dim, generator=g, device="cuda") for _ in range(2))
    rng = torch.tensor([1, 2], dtype=torch.int64, device="cuda")
    want = (tp.tp_norm_fwd(norm, x), *tp.tp_norm_bwd(norm, x, gy), tp.tp_dropout_fwd(drop, x, 0.3, rng))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        got = (tp.tp_norm_fwd(norm, x, stream=stream), *tp.tp_norm_bwd(norm, x, gy, stream=stream),
               tp.tp_dropout_fwd(drop, x, 0.3, rng, stream=stream))
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_device_memory_with_buffers_given(tp):
    """With outputs and workspaces given, no call allocates."""
    P, rowptr, src, vec, x, gy = _make_layer(tp, seed=5)
    N, E = 40, len(src)
    rowptr, src, vec = dev(rowptr), dev(src), dev(vec)
    new = lambda *s: torch.empty(*s, device="cuda")
    byte = lambda n: torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
    rng = torch.tensor([3, 4], dtype=torch.int64, device="cuda")
    attn, norm, drop = P["attn"], P["norm"], P["drop"]
    ws_f, ws_b = byte(tp.tp_attn_workspace_size(attn, N, E, 0)), byte(tp.tp_attn_workspace_size(attn, N, E, 1))
    ws_n = byte(tp.tp_norm_workspace_size(norm, N, 1))
    bucket, y, lse, z = torch.empty(E, dtype=torch.int32, device="cuda"), new(N, 40), new(N, HEADS), new(N, 40)
    gq, gk, gv, gt, gw, gb = new(N, 40), new(N, 40), new(N, 40), new(K, HEADS), new(24), new(16)

    def step():
        tp.tp_distance_buckets(vec, P["bounds"], 2.5, bucket=bucket)
        tp.tp_norm_fwd(norm, x, P["weight"], P["bias"], y=z)
        more = dict(bucket=bucket, table=P["table"], p=0.2, rng=rng)
        tp.tp_attn_fwd(attn, rowptr, src, z, z, z, y=y, lse=lse, ws=ws_f, **more)
        tp.tp_attn_bwd(attn, rowptr, src, z, z, z, y, lse, gy, gq=gq, gk=gk, gv=gv, gtable=gt, ws=ws_b, **more)
        tp.tp_norm_bwd(norm, x, gq, P["weight"], gx=gq, gweight=gw, gbias=gb, ws=ws_n)
        tp.tp_dropout_fwd(drop, y, 0.2, rng, y=y)
    step()
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before, free = torch.cuda.memory_allocated(), torch.cuda.mem_get_info()[0]
    step()
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() == before and torch.cuda.mem_get_info()[0] == free


@pytest.mark.parametrize("irreps", ["16x0e+8x1o", "7x0e+5x1o", "1201x0e"])
def test_norm_with_the_smallest_eps(tp, irreps):
    """Zero rows stay zero and rows of squares below the smallest normal float are as good as their eps allows."""
    norm, rng = tp.Norm(irreps, 1.1e-30), np.random.default_rng(0)
    x = rng.standard_normal((6, norm.dim)).astype(np.float32)
    x[0], x[1:] = 0, x[1:] * np.array([1e-15, 1e-17, 1e-19, 1e-20, 1.0], np.float32)[:, None]
    y = tp.tp_norm_fwd(norm, dev(x))
    assert bool((y[0] == 0).all())
    eps = float(np.float32(1.1e-30))
    bound = norm_bounds(irreps, x, None, None, x, eps)["y"]
    want = oa.norm(irreps, x, eps=eps)
    # every flushed square takes at most 2^-126 from the mean square, 2^-27 of eps
    assert_within(y, want, bound + 2.0 ** -27 * np.abs(want.numpy()), "y")


@pytest.mark.parametrize("irreps,rows", [("1x0e", 4736), ("1x0e", 4737), ("3x1o", 30011), ("1x0e", 120001), ("2x0e", 500009), ("7x0e+5x1o", 30011),
                                         ("4x0e+4x1o", 120001), ("5x0o", 7105), ("32x0e+32x1o", 14209), ("31x0e+31x1o", 4737),
                                         ("128x0e", 30011), ("32x0e+32x1o+32x2e", 9473), ("33x0e+33x1o", 20001), ("129x0e", 9471)])
def test_dropout_of_many_rows(tp, irreps, rows):
    """Several narrow rows a warp, tiles that end short, and more rows than warps."""
    import attn_fast
    drop, rng = tp.Dropout(irreps), np.random.default_rng(rows)
    x = rng.standard_normal((rows, drop.dim)).astype(np.float32)
    seed, offset, site, p = 11, 1 << 35, 2, 0.3
    r = torch.tensor([seed, offset], dtype=torch.int64, device="cuda")
    y = tp.tp_dropout_fwd(drop, dev(x), p, r, site)
    keep = attn_fast.keep_values(seed, offset + site, rows * drop.n_channels, p).reshape(rows, -1)
    ir = Irreps(irreps)
    want = x.astype(np.float64) * np.concatenate([np.repeat(keep[:, c:c + mul], 2 * l + 1, 1)
                                                  for (mul, l, _), c in zip(ir.blocks, np.cumsum([0] + [m for m, _, _ in ir.blocks]))], 1)
    # one rounding of 1/(1-p) and one of the product
    assert_within(y, torch.as_tensor(want), 2 * U * np.abs(want) * (1 + 2 * U), "y")
    assert torch.equal(y == 0, dev(want) == 0)
    own = dev(x)
    assert tp.tp_dropout_fwd(drop, own, p, r, site, y=own) is own and torch.equal(own, y)
    buf = torch.full((rows * drop.dim + 2,), 5.0, device="cuda")
    tp.tp_dropout_fwd(drop, dev(x), p, r, site, y=buf[1:-1].view(rows, drop.dim))
    assert torch.equal(buf[1:-1].view(rows, drop.dim), y) and float(buf[0]) == 5.0 and float(buf[-1]) == 5.0


def test_layer_gradient_against_differences_of_its_own_forward(tp):
    P, rowptr, src, vec, x, gy = _make_layer(tp, seed=1)
    x.requires_grad_(True)
    graph, rng = tp.autograd.Graph(dev(rowptr), dev(src)), torch.tensor([3, 4], dtype=torch.int64, device="cuda")
    y = _layer(tp, P, x, graph, dev(vec), rng, 0.2)
    (gx,) = torch.autograd.grad(y, x, gy)
    step, eps = torch.randn(x.shape, generator=torch.Generator().manual_seed(1)).cuda(), 2.0 ** -5
    dot = lambda a, b: float((a.double() * b.double()).sum())
    with torch.no_grad():
        ends = [x + s * eps * step for s in (1, -1)]
        own = dot(_layer(tp, P, ends[0], graph, dev(vec), rng, 0.2).double() - _layer(tp, P, ends[1], graph, dev(vec), rng, 0.2).double(), gy)
        exact = [_oracle_layer(P, a, rowptr, src, vec, 0.2, 3, 4)[0].detach() for a in ends]
    want_y, want_x, _ = _oracle_layer(P, x, rowptr, src, vec, 0.2, 3, 4)
    (want,) = torch.autograd.grad(want_y, want_x, gy.double().cpu())
    # the quotient is off by its truncation, which the same quotient in 64 bits tells, and by the roundings of two
    # forward passes: sums of at most 24 terms in four operators, 64 u of the largest output each
    truncation = abs(dot(exact[0] - exact[1], gy.cpu()) / (2 * eps) - dot(want, step.cpu()))
    rounding = 2 * float(gy.abs().sum()) * 64 * U * float(y.detach().abs().max()) / (2 * eps)
    assert truncation + rounding <= 0.1 * float(gx.norm())     # the size of a derivative along a random direction
    assert abs(own / (2 * eps) - dot(gx, step)) <= truncation + rounding
