"""Host-side checks of graph attention, the distance buckets, the norm and the dropout
(include/tp_attn.h, include/tp_block.h), no GPU needed: sizes, refusals before anything reaches
the device, and no CPU path."""
import ctypes as C
import math
import os
import subprocess
import sys

import pytest
import torch

from oracle.irreps import Irreps


@pytest.fixture(scope="module")
def tp():
    from equivariant_tensor_product_b200 import build
    build.build()
    import equivariant_tensor_product_b200 as tp
    return tp


def test_sizes(tp):
    for qk, v, heads in (("4x0e+4x1o", "4x0e+4x1o", 2), ("64x0e", "32x0e+32x1o+32x2e+32x3o", 8), ("21x0e", "21x2e+3x3o", 3)):
        a = tp.Attention(qk, v, heads, 7)
        assert (a.qk_dim, a.v_dim) == (Irreps(qk).dim, Irreps(v).dim)
    n = tp.Norm("3x0e+2x0o+4x1o+5x0e")
    assert (n.dim, n.n_weights, n.n_bias) == (22, 14, 8)
    d = tp.Dropout("3x0e+2x0o+4x1o+5x0e")
    assert (d.dim, d.n_channels) == (22, 14)


def test_workspace_holds_no_edge_feature_tensor(tp):
    a = tp.Attention("128x0e+128x1o+128x2e", "128x0e+128x1o+128x2e", 8, 32)
    N, E = 100000, 3001138
    bwd = tp.tp_attn_workspace_size(a, N, E, tp.TP_OP_BWD)
    # two floats per edge and head, receiver, sender order and its scratch, and node-sized partials
    assert bwd <= E * (8 * 8 + 4 + 4 + 12) + 8 * N * a.v_dim + (64 << 20)
    assert tp.tp_attn_workspace_size(a, N, E, tp.TP_OP_FWD) <= 4 * N * a.v_dim + (1 << 20)
    assert tp.tp_attn_workspace_size(a, 24, 192, tp.TP_OP_FWD) == 0
    n = tp.Norm("128x0e+128x1o+128x2e")
    assert tp.tp_norm_workspace_size(n, 100000, tp.TP_OP_FWD) == 0
    assert tp.tp_norm_workspace_size(n, 100000, tp.TP_OP_BWD) <= 8 * n.dim * 148 * 8


@pytest.mark.parametrize("args,status", [
    (("4x0e", "4x0e", 0), 1), (("4x0e", "4x0e", 3), 1), (("4x0e", "6x0e", 4), 1), (("4x0e+", "4x0e", 1), 1),
    (("", "4x0e", 1), 1), (("4x4e", "4x0e", 1), 2), (("64x0e", "64x0e", 64), 2), (("4x0e", "4x0e", 1, -1), 1),
    (("4x0e", "4x0e", 1, 5000), 2), (("32x0e", "32x0e", 32, 2000), 2), (("5000x0e", "4x0e", 1), 2),
    (("4x0e", "600x3o", 1), 2), (("+".join(["1x0e"] * 17), "4x0e", 1), 2),
])
def test_attention_validation(tp, args, status):
    with pytest.raises(tp.TPError) as e:
        tp.Attention(*args)
    assert e.value.status == status


@pytest.mark.parametrize("make,status", [
    (lambda tp: tp.Norm("4x0e+"), 1), (lambda tp: tp.Norm("4x4e"), 2), (lambda tp: tp.Norm("9000x0e"), 2),
    (lambda tp: tp.Norm("4x0e", 0.0), 1), (lambda tp: tp.Norm("4x0e", -1.0), 1), (lambda tp: tp.Norm("4x0e", math.nan), 1),
    (lambda tp: tp.Norm("4x0e", math.inf), 1), (lambda tp: tp.Dropout("0x0e"), 1), (lambda tp: tp.Dropout("4x4o"), 2),
    (lambda tp: tp.Dropout("9999999x3o"), 2), (lambda tp: tp.Norm("+".join(["1x0e"] * 17)), 2),
])
def test_norm_and_dropout_validation(tp, make, status):
    with pytest.raises(tp.TPError) as e:
        make(tp)
    assert e.value.status == status


FAKE, ODD, BIG = C.c_void_p(0x10000), C.c_void_p(0x10002), 1 << 30     # never touched: every call fails host checks


def _fwd(lib, h, N=4, E=8, rowptr=FAKE, src=FAKE, bucket=FAKE, q=FAKE, ldq=16, k=FAKE, ldk=16, v=FAKE, ldv=16, table=FAKE,
         scale=1.0, p=0.0, rng=None, site=0, y=FAKE, lse=FAKE, ws=FAKE, size=BIG):
    return lib.tp_attn_fwd(h, N, E, rowptr, src, bucket, q, ldq, k, ldk, v, ldv, table, scale, p, rng, site, y, lse, ws, size,
                           None)


def _bwd(lib, h, N=4, E=8, rowptr=FAKE, src=FAKE, colptr=FAKE, perm=FAKE, bucket=FAKE, q=FAKE, ldq=16, k=FAKE, ldk=16,
         v=FAKE, ldv=16, table=FAKE, scale=1.0, p=0.0, rng=None, site=0, y=FAKE, lse=FAKE, gy=FAKE, gq=FAKE, ldgq=16,
         gk=FAKE, ldgk=16, gv=FAKE, ldgv=16, gtable=FAKE, ws=FAKE, size=BIG):
    return lib.tp_attn_bwd(h, N, E, rowptr, src, colptr, perm, bucket, q, ldq, k, ldk, v, ldv, table, scale, p, rng, site, y,
                           lse, gy, gq, ldgq, gk, ldgk, gv, ldgv, gtable, ws, size, None)


def test_attention_calls_reject_bad_arguments_before_the_device(tp):
    lib = tp.load()
    a, plain = tp.Attention("4x0e+4x1o", "4x0e+4x1o", 2, 5), tp.Attention("4x0e+4x1o", "4x0e+4x1o", 2)
    h = a.handle
    for call in (_fwd, _bwd):
        assert call(lib, None) == 1
        assert call(lib, h, N=-1) == 1 and call(lib, h, E=-1) == 1
        assert call(lib, h, N=1 << 30) == 2 and call(lib, h, E=1 << 31) == 2
        for name in ("rowptr", "src", "q", "k", "v"):
            assert call(lib, h, **{name: None}) == 1
            assert call(lib, h, **{name: ODD}) == 1
        for name in ("ldq", "ldk", "ldv"):
            assert call(lib, h, **{name: 15}) == 1
        assert call(lib, h, table=FAKE, bucket=None) == 1
        assert call(lib, plain.handle) == 1                                   # buckets without a table's size
        assert call(lib, h, scale=math.nan) == 1 and call(lib, h, scale=math.inf) == 1
        for p in (-0.1, 1.0, math.nan, 1.0 - 2.0 ** -40):
            assert call(lib, h, p=p, rng=FAKE) == 1
        assert call(lib, h, p=0.5, rng=None) == 1
        assert call(lib, h, p=0.5, rng=C.c_void_p(0x10004)) == 1              # rng is 64-bit
    assert _fwd(lib, h, y=None) == 1 and _fwd(lib, h, y=ODD) == 1 and _fwd(lib, h, lse=ODD) == 1
    assert _fwd(lib, h, N=0, rowptr=None, q=None) == 0
    for name in ("y", "lse", "gy"):
        assert _bwd(lib, h, **{name: None}) == 1 and _bwd(lib, h, **{name: ODD}) == 1
    for name in ("gq", "gk", "gv", "gtable", "colptr", "perm"):
        assert _bwd(lib, h, **{name: ODD}) == 1
    assert _bwd(lib, h, colptr=None) == 1 and _bwd(lib, h, perm=None) == 1
    assert _bwd(lib, h, ldgq=15) == 1 and _bwd(lib, h, ldgk=15) == 1 and _bwd(lib, h, ldgv=15) == 1
    assert _bwd(lib, h, table=None) == 1                                      # gtable of no table
    assert _bwd(lib, plain.handle, bucket=None, table=None) == 1
    assert _bwd(lib, h, size=1024) == 4 and _bwd(lib, h, ws=None) == 4 and _bwd(lib, h, ws=C.c_void_p(0x10040)) == 4
    assert _bwd(lib, h, gq=None, gk=None, gv=None, gtable=None) == 0
    size = C.c_size_t()
    assert lib.tp_attn_workspace_size(h, 4, 8, 2, C.byref(size)) == 1         # first order only
    assert lib.tp_attn_workspace_size(None, 4, 8, 0, C.byref(size)) == 1
    assert lib.tp_attn_create(None, b"4x0e", b"4x0e", 1, 0) == 1
    assert lib.tp_attn_create(C.byref(C.c_void_p()), None, b"4x0e", 1, 0) == 1


def test_bucket_norm_and_dropout_calls_reject_bad_arguments(tp):
    lib = tp.load()
    b = lib.tp_distance_buckets
    assert b(-1, FAKE, 3, FAKE, 5.0, FAKE, None) == 1 and b(4, FAKE, -1, FAKE, 5.0, FAKE, None) == 1
    assert b(4, FAKE, 1024, FAKE, 5.0, FAKE, None) == 2
    assert b(4, FAKE, 3, FAKE, -1.0, FAKE, None) == 1 and b(4, FAKE, 3, FAKE, math.nan, FAKE, None) == 1
    assert b(4, None, 3, FAKE, 5.0, FAKE, None) == 1 and b(4, FAKE, 3, None, 5.0, FAKE, None) == 1
    assert b(4, FAKE, 3, FAKE, 5.0, ODD, None) == 1 and b(0, None, 3, None, 5.0, None, None) == 0
    n, d = tp.Norm("4x0e+4x1o"), tp.Dropout("4x0e+4x1o")
    f = lib.tp_norm_fwd
    assert f(None, 4, FAKE, FAKE, FAKE, FAKE, None) == 1 and f(n.handle, -1, FAKE, FAKE, FAKE, FAKE, None) == 1
    assert f(n.handle, 4, None, FAKE, FAKE, FAKE, None) == 1 and f(n.handle, 4, FAKE, FAKE, FAKE, None, None) == 1
    assert f(n.handle, 4, FAKE, ODD, FAKE, FAKE, None) == 1 and f(n.handle, 1 << 41, FAKE, FAKE, FAKE, FAKE, None) == 2
    assert f(n.handle, 0, None, None, None, None, None) == 0
    g = lib.tp_norm_bwd
    assert g(None, 4, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, BIG, None) == 1
    assert g(n.handle, 4, None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, BIG, None) == 1
    assert g(n.handle, 4, FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, BIG, None) == 1
    assert g(n.handle, 4, FAKE, FAKE, FAKE, ODD, FAKE, FAKE, FAKE, BIG, None) == 1
    assert g(n.handle, 4, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 16, None) == 4
    assert g(n.handle, 4, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, 0, None) == 4
    assert g(n.handle, 4, FAKE, FAKE, FAKE, None, None, None, None, 0, None) == 0
    size = C.c_size_t()
    assert lib.tp_norm_workspace_size(n.handle, 4, 2, C.byref(size)) == 1
    for call in (lib.tp_dropout_fwd, lib.tp_dropout_bwd):
        assert call(None, 4, FAKE, 0.5, FAKE, 0, FAKE, None) == 1
        assert call(d.handle, 4, FAKE, 1.0, FAKE, 0, FAKE, None) == 1
        assert call(d.handle, 4, FAKE, 0.5, None, 0, FAKE, None) == 1
        assert call(d.handle, 4, None, 0.5, FAKE, 0, FAKE, None) == 1
        assert call(d.handle, 4, FAKE, 0.5, FAKE, 0, ODD, None) == 1
        assert call(d.handle, 4, FAKE, 0.5, C.c_void_p(0x10004), 0, FAKE, None) == 1
        assert call(d.handle, -4, FAKE, 0.5, FAKE, 0, FAKE, None) == 1
        assert call(d.handle, 0, None, 0.5, FAKE, 0, None, None) == 0
    assert lib.tp_norm_create(None, b"4x0e", 1e-5) == 1 and lib.tp_dropout_create(None, b"4x0e") == 1
    assert lib.tp_last_error_message()


def test_binding_refuses_what_it_cannot_pass_on(tp):
    """Shapes, devices and strides are refused in Python; no CPU tensor goes any further."""
    a = tp.Attention("4x0e+4x1o", "4x0e+4x1o", 2, 5)
    rowptr, src = torch.tensor([0, 1, 2], dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(2, 16)
    with pytest.raises(ValueError, match="CUDA"):
        tp.tp_attn_fwd(a, rowptr, src, x, x, x)
    with pytest.raises(ValueError, match="shape"):
        tp.tp_attn_fwd(a, rowptr, src, x, x[:, :12], x)
    with pytest.raises(ValueError, match="table must have shape"):
        tp.tp_attn_fwd(a, rowptr, src, x, x, x, bucket=src, table=torch.zeros(4, 2))
    with pytest.raises(ValueError, match="bucket must have shape"):
        tp.tp_attn_fwd(a, rowptr, src, x, x, x, bucket=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="both"):
        tp.tp_attn_bwd(a, rowptr, src, x, x, x, x, torch.zeros(2, 2), x, colptr=rowptr)
    with pytest.raises(ValueError, match="CUDA"):
        tp.tp_distance_buckets(torch.zeros(2, 3), torch.ones(1), 5.0)
    with pytest.raises(ValueError, match="shape"):
        tp.tp_distance_buckets(torch.zeros(2, 4), torch.ones(1), 5.0)
    n, d = tp.Norm("4x0e+4x1o"), tp.Dropout("4x0e+4x1o")
    with pytest.raises(ValueError, match="shape"):
        tp.tp_norm_fwd(n, torch.zeros(2, 15))
    with pytest.raises(ValueError, match="weight must have shape"):
        tp.tp_norm_fwd(n, x, torch.zeros(4))
    with pytest.raises(ValueError, match="shape"):
        tp.tp_dropout_fwd(d, torch.zeros(2, 15), 0.0)
    from equivariant_tensor_product_b200._marshal import rows
    meta = torch.zeros(4, 16)
    with pytest.raises(ValueError):
        rows(meta.t(), 0, 16, 4, "q")


def test_no_cpu_path_without_a_device(tp):
    if torch.cuda.is_available():
        pytest.skip("device present")
    lib = tp.load()
    assert _fwd(lib, tp.Attention("4x0e+4x1o", "4x0e+4x1o", 2, 5).handle) == 5
    assert _bwd(lib, tp.Attention("4x0e+4x1o", "4x0e+4x1o", 2, 5).handle) == 5
    assert lib.tp_norm_fwd(tp.Norm("4x0e").handle, 4, FAKE, FAKE, FAKE, FAKE, None) == 5
    assert lib.tp_dropout_fwd(tp.Dropout("4x0e").handle, 4, FAKE, 0.5, FAKE, 0, FAKE, None) == 5
    assert lib.tp_distance_buckets(4, FAKE, 3, FAKE, 5.0, FAKE, None) == 5


def test_norm_on_one_handle_from_two_threads(tp, monkeypatch):
    """Between a backward call's look at the handle's workspace size and its use, another thread's call with
    other rows may change it."""
    from equivariant_tensor_product_b200 import block
    asked = []

    class Handle:
        dim, n_weights, n_bias, handle = 4, 4, 4, None
        looks = 0

        class _lib:
            tp_norm_bwd = staticmethod(lambda *a: 0)

        @property
        def _size(self):
            self.looks += 1
            return (3, 48) if self.looks == 1 else (1000, 16000)

        @_size.setter
        def _size(self, value):
            pass
    monkeypatch.setattr(block, "device_index", lambda t, name: 0)
    monkeypatch.setattr(block, "on", lambda i, stream: torch.no_grad())
    monkeypatch.setattr(block, "f32", lambda *a: None)
    monkeypatch.setattr(block, "stream_of", lambda i: 0)
    monkeypatch.setattr(block, "workspace", lambda ws, need, i: asked.append(need) or (None, None, need))
    monkeypatch.setattr(block, "tp_norm_workspace_size", lambda norm, N, op: 16 * N)
    x = torch.zeros(3, 4)
    tp.tp_norm_bwd(Handle(), x, x)
    assert asked == [48]


def test_import_needs_no_cuda_build_of_torch(tp):
    """Plans, their sizes and refusals are host code: a torch without CUDA lacks the raw-stream function."""
    code = ("import torch; del torch._C._cuda_getCurrentRawStream; import equivariant_tensor_product_b200 as tp; "
            "print(tp.Norm('4x0e+4x1o').dim)")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=os.path.dirname(os.path.dirname(__file__)))
    assert r.returncode == 0 and r.stdout.split() == ["16"], r.stderr[-2000:]


def test_norm_refuses_an_eps_that_squares_in_32_bits_cannot_stand_beside(tp):
    """Squares below 2^-126 are flushed to zero: beside an eps near it they would be missing from the mean square,
    and an eps below it is zero itself, which makes a NaN of a zero row."""
    for eps in (1e-45, 1e-40, 1e-38, 9e-31):
        with pytest.raises(tp.TPError) as e:
            tp.Norm("4x0e+4x1o", eps)
        assert e.value.status == 1
    tp.Norm("4x0e+4x1o", 1.1e-30)


def test_outputs_may_not_start_where_inputs_do(tp):
    from equivariant_tensor_product_b200._marshal import apart
    apart((16, None, 64), (None, 32, 48), "outputs")
    apart((None, None), (None, 32), "outputs")
    for outputs, inputs in (((16, 32), (32, 48)), ((16, 16), (32, 48)), ((None, 48), (None, 48))):
        with pytest.raises(ValueError, match="share memory"):
            apart(outputs, inputs, "outputs")


def test_rows_are_refused_for_their_strides(tp):
    """The device index of CPU tensors is -1: with it the check of the strides is reached."""
    from equivariant_tensor_product_b200._marshal import rows
    for bad in (torch.zeros(4, 16).t(), torch.zeros(1, 4).expand(16, 4), torch.zeros(16, 8)[:, ::2]):
        with pytest.raises(ValueError, match="contiguous rows"):
            rows(bad, -1, 16, 4, "q")
    wide = torch.zeros(16, 8)
    assert rows(wide[:, 4:], -1, 16, 4, "q") == (wide.data_ptr() + 16, 8)
