"""Pins of the float64 forms in oracle/attn.py: a pure-Python loop, rotation and inversion
equivariance, dense softmax attention as a special case, finite differences, the published test
vectors of the generator, scipy/numpy special cases of the norm, and planted mistakes."""
import math

import numpy as np
import pytest
import torch

from oracle import attn as oa
from oracle.irreps import Irreps
from oracle.so3 import random_rotation, wigner_D

QK, V, H = "4x0e+4x1o", "6x0e+4x1o+2x2e", 2


def _graph(seed=0, n=7, deg=4):
    rng = np.random.default_rng(seed)
    counts = rng.integers(0, 2 * deg, n)
    counts[2] = 0
    rowptr = np.concatenate([[0], np.cumsum(counts)])
    src = rng.integers(0, n, rowptr[-1])
    bucket = rng.integers(-1, 3, rowptr[-1])
    return rowptr, src, bucket


def _inputs(seed=0):
    rng = np.random.default_rng(seed)
    rowptr, src, bucket = _graph(seed)
    n = len(rowptr) - 1
    f = lambda *s: rng.standard_normal(s)
    return dict(rowptr=rowptr, src=src, q=f(n, Irreps(QK).dim), k=f(n, Irreps(QK).dim), v=f(n, Irreps(V).dim),
                bucket=bucket, table=f(3, H), n_buckets=3, scale=0.4), f(n, Irreps(V).dim)


def test_attention_against_a_loop_over_single_floats():
    d, _ = _inputs()
    y, lse = oa.attention(QK, V, H, **d)
    N = len(d["rowptr"]) - 1
    qk_cols = {0: [0, 1] + list(range(4, 10)), 1: [2, 3] + list(range(10, 16))}
    v_cols = {0: [0, 1, 2] + list(range(6, 12)) + list(range(18, 23)),
              1: [3, 4, 5] + list(range(12, 18)) + list(range(23, 28))}
    for i in range(N):
        for h in range(H):
            es = [e for e in range(d["rowptr"][i], d["rowptr"][i + 1]) if d["bucket"][e] >= 0]
            s = [d["scale"] * sum(d["q"][i][c] * d["k"][d["src"][e]][c] for c in qk_cols[h]) + d["table"][d["bucket"][e]][h]
                 for e in es]
            z = sum(math.exp(t) for t in s)
            for c in v_cols[h]:
                want = sum(math.exp(t) / z * d["v"][d["src"][e]][c] for t, e in zip(s, es)) if es else 0.0
                assert abs(float(y[i, c]) - want) < 1e-12
            assert (float(lse[i, h]) == -math.inf) if not es else abs(float(lse[i, h]) - math.log(z)) < 1e-12


def test_full_graph_is_dense_softmax_attention():
    n, rng = 5, np.random.default_rng(3)
    q, k, v = (rng.standard_normal((n, 8)) for _ in range(3))
    rowptr, src = np.arange(n + 1) * n, np.tile(np.arange(n), n)
    y, lse = oa.attention("8x0e", "8x0e", 1, rowptr, src, q, k, v, scale=0.3)
    s = 0.3 * q @ k.T
    p = np.exp(s) / np.exp(s).sum(1, keepdims=True)
    np.testing.assert_allclose(y.numpy(), p @ v, atol=1e-12)
    np.testing.assert_allclose(lse.numpy()[:, 0], np.log(np.exp(s).sum(1)), atol=1e-12)


def _rotate(irreps, x, R, inversion):
    ir, out = Irreps(irreps), []
    for (mul, l, p), off in zip(ir.blocks, ir.offsets):
        b = torch.as_tensor(x)[:, off:off + mul * (2 * l + 1)].reshape(-1, mul, 2 * l + 1)
        D = torch.as_tensor(np.asarray(wigner_D(l, R)), dtype=torch.float64)
        out.append((torch.einsum("ab,nub->nua", D, b.double()) * (p if inversion else 1)).reshape(len(x), -1))
    return torch.cat(out, 1)


@pytest.mark.parametrize("inversion", [False, True])
def test_attention_and_norm_are_equivariant(inversion):
    d, _ = _inputs(1)
    R = random_rotation(np.random.default_rng(5))
    turned = dict(d, q=_rotate(QK, d["q"], R, inversion), k=_rotate(QK, d["k"], R, inversion),
                  v=_rotate(V, d["v"], R, inversion))
    y, lse = oa.attention(QK, V, H, **d)
    y2, lse2 = oa.attention(QK, V, H, **turned)
    np.testing.assert_allclose(y2.numpy(), _rotate(V, y.numpy(), R, inversion).numpy(), atol=1e-10)
    np.testing.assert_allclose(lse2.numpy(), lse.numpy(), atol=1e-10)
    ir = "3x0e+2x0o+2x1o+3x2e"
    rng = np.random.default_rng(0)
    x, w, b = rng.standard_normal((4, Irreps(ir).dim)), rng.standard_normal(10), rng.standard_normal(3)
    np.testing.assert_allclose(oa.norm(ir, _rotate(ir, x, R, inversion), w, b).numpy(),
                               _rotate(ir, oa.norm(ir, x, w, b).numpy(), R, inversion).numpy(), atol=1e-10)


def test_gradients_against_finite_differences():
    d, gy = _inputs(2)
    r = np.random.default_rng(9).choice([0.0, 1.25], size=(len(d["src"]), H), p=[0.2, 0.8])
    g = oa.attention_backward(QK, V, H, gy=gy, r=r, **d)
    f = lambda **kw: float((oa.attention(QK, V, H, r=r, **dict(d, **kw))[0] * torch.as_tensor(gy)).sum())
    for name in ("q", "k", "v", "table"):
        rng = np.random.default_rng(4)
        step = rng.standard_normal(d[name].shape)
        eps = 1e-6
        num = (f(**{name: d[name] + eps * step}) - f(**{name: d[name] - eps * step})) / (2 * eps)
        assert abs(num - float((g["g" + name] * torch.as_tensor(step)).sum())) < 1e-6
    ir, rng = "3x0e+2x0o+2x1o", np.random.default_rng(5)
    x, w, b, gy = rng.standard_normal((5, 11)), rng.standard_normal(7), rng.standard_normal(3), rng.standard_normal((5, 11))
    g = oa.norm_backward(ir, x, gy, w, b)
    f = lambda x_, w_, b_: float((oa.norm(ir, x_, w_, b_) * torch.as_tensor(gy)).sum())
    for i, name in enumerate(("gx", "gweight", "gbias")):
        step = rng.standard_normal([x, w, b][i].shape)
        hi, lo = [x, w, b], [x, w, b]
        hi[i], lo[i] = hi[i] + 1e-6 * step, lo[i] - 1e-6 * step
        assert abs((f(*hi) - f(*lo)) / 2e-6 - float((g[name] * torch.as_tensor(step)).sum())) < 1e-6


def test_generator_has_the_published_test_vectors():
    # the known answers that the generator's authors publish for philox4x32-10
    assert [hex(int(w)) for w in oa.philox_words(0, 0, 4)] == ["0x6627e8d5", "0xe169c58d", "0xbc57ac4c", "0x9b00dbd8"]
    words = oa.philox_words(0, 0, 11)
    assert len(words) == 11 and len(set(words.tolist())) == 11
    np.testing.assert_array_equal(oa.philox_words(5, 7, 3), oa.philox_words(5, 7, 40)[:3])
    assert (oa.philox_words(5, 7, 8) != oa.philox_words(5, 8, 8)).all()
    keep = oa.keep_values(11, 13, 20000, 0.25)
    # 20,000 draws of probability 1/4: six standard deviations are 0.0184
    assert abs((keep == 0).mean() - 0.25) < 0.0184 and set(np.unique(keep)) == {0.0, 1.0 / 0.75}


def test_norm_special_cases():
    rng = np.random.default_rng(0)
    x, w, b = rng.standard_normal((6, 16)), rng.standard_normal(16), rng.standard_normal(16)
    want = torch.nn.functional.layer_norm(torch.as_tensor(x), (16,), torch.as_tensor(w), torch.as_tensor(b), 1e-5)
    np.testing.assert_allclose(oa.norm("16x0e", x, w, b).numpy(), want.numpy(), atol=1e-12)
    y = oa.norm("4x1o", x[:, :12], eps=1e-12).numpy()
    np.testing.assert_allclose((y ** 2).mean(1), 1.0, atol=1e-9)          # unit mean square, direction kept
    np.testing.assert_allclose(y / x[:, :12], (y / x[:, :12])[:, :1].repeat(12, 1), rtol=1e-9)


def test_buckets_and_dropout_special_cases():
    bounds = [0.5, 1.0, 2.0]
    vec = [[0, 0, 0], [0.5, 0, 0], [0, 0.75, 0], [0, 0, 1.0], [3, 0, 0], [0, 5, 0], [math.nan, 0, 0]]
    assert oa.distance_buckets(vec, bounds, 5.0).tolist() == [0, 1, 1, 2, 3, -1, -1]
    assert oa.distance_buckets(vec, bounds).tolist() == [0, 1, 1, 2, 3, 3, -1]
    x = np.ones((50, 2 + 6))
    y = oa.dropout("2x0e+2x1o", x, 0.5, 3, 4).numpy()
    assert set(np.unique(y)) == {0.0, 2.0}
    assert (y[:, 2:5] == y[:, 2:3]).all() and (y[:, 5:8] == y[:, 5:6]).all()


def test_planted_mistakes_are_caught():
    """A softmax over the wrong edges, a head layout that splits the row instead of the channels and a mean
    taken off an odd block each break a pin above."""
    d, _ = _inputs()
    y, _ = oa.attention(QK, V, H, **d)
    wrong = dict(d, bucket=np.maximum(d["bucket"], 0))                     # masked edges let in
    assert float((oa.attention(QK, V, H, **wrong)[0] - y).abs().max()) > 1e-3
    R = random_rotation(np.random.default_rng(5))
    halves = [np.arange(8), np.arange(8, 16)]                              # the row cut in two
    s = lambda q, k: float(q[halves[0]] @ k[halves[0]])
    q, k = d["q"], d["k"]
    q2, k2 = _rotate(QK, q, R, False).numpy(), _rotate(QK, k, R, False).numpy()
    assert abs(s(q[0], k[1]) - s(q2[0], k2[1])) > 1e-3
    x = np.random.default_rng(1).standard_normal((3, 4))
    mean_off = x - x.mean(1, keepdims=True)
    odd = oa.norm("4x0o", x).numpy()
    wrong = mean_off / np.sqrt((mean_off ** 2).mean(1, keepdims=True) + 1e-5)
    assert np.abs(odd - wrong).max() > 1e-2
