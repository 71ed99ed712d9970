"""The norm, int8 product and sorted-row operators without a GPU: host checks of every entry point, the
gradient formulas against differences and against automatic differentiation, and their workspace size."""

import ctypes as C
import os
import subprocess

import pytest
import torch

from grouped_gemm_02_b200 import build, moe
from tests import ops_helpers as R

P = C.c_void_p(0x10000)          # never dereferenced: every call below ends in its host checks
ODD = C.c_void_p(0x10008)


@pytest.fixture(scope="module")
def L():
    build.build()
    return moe.lib()


def _norm(L, name, **kw):
    a = dict(x=P, residual=None, weight=P, T=4, d=256, eps=1e-6, xsum=None, y=P, q=P, scale=P)
    a.update(kw)
    args = [a[n] for n in ("x", "residual", "weight", "T", "d", "eps", "xsum", "y")]
    if name != "moe_rmsnorm":
        args += [a["q"], a["scale"]]
    return getattr(L, name)(*args, None)


@pytest.mark.parametrize("name", ["moe_rmsnorm", "moe_rmsnorm_fp8", "moe_rmsnorm_int8"])
def test_norm_refusals(L, name):
    assert _norm(L, name, T=0) == 0
    assert _norm(L, name, T=-1) == -1
    assert _norm(L, name, T=1 << 31) == -1
    assert _norm(L, name, d=0) == -1
    assert _norm(L, name, d=32768 + 128) == -1
    assert _norm(L, name, d=96) == -2
    assert _norm(L, name, d=192, x=None) == (-2 if name == "moe_rmsnorm_fp8" else -1)
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        assert _norm(L, name, eps=eps) == -1
    assert _norm(L, name, x=None) == -1
    assert _norm(L, name, weight=None) == -1
    assert _norm(L, name, residual=P) == -1                  # a residual without a place for the sum
    assert _norm(L, name, xsum=P) == -1                      # a place for the sum without a residual
    assert _norm(L, name, residual=P, xsum=ODD) == -2
    assert _norm(L, name, residual=ODD, xsum=P) == -2
    assert _norm(L, name, x=ODD) == -2
    assert _norm(L, name, weight=ODD) == -2
    assert _norm(L, name, y=ODD) == -2
    if name == "moe_rmsnorm":
        assert _norm(L, name, y=None) == -1
    else:
        assert _norm(L, name, q=None) == -1
        assert _norm(L, name, scale=None) == -1
        assert _norm(L, name, q=ODD) == -2


def _norm_grad(L, **kw):
    a = dict(dy=P, xsum=P, weight=P, dxsum=None, T=4, d=256, eps=1e-6, dx=P, dweight=P, ws=P, ws_bytes=1 << 30)
    a.update(kw)
    return L.moe_rmsnorm_backward(*[a[n] for n in ("dy", "xsum", "weight", "dxsum", "T", "d", "eps", "dx", "dweight",
                                                   "ws", "ws_bytes")], None)


def test_norm_grad_refusals(L):
    assert _norm_grad(L, T=-1) == -1
    assert _norm_grad(L, d=32832) == -1
    assert _norm_grad(L, d=100) == -2
    assert _norm_grad(L, eps=0.0) == -1
    for name in ("dy", "xsum", "weight", "dx", "dweight", "ws"):
        assert _norm_grad(L, **{name: None}) == -1, name
    for name in ("dy", "xsum", "weight", "dxsum", "dx", "dweight", "ws"):
        assert _norm_grad(L, **{name: ODD}) == -2, name
    need = moe.moe_rmsnorm_backward_workspace_size(4, 256)
    assert _norm_grad(L, ws_bytes=need // 2) == -3


@pytest.mark.parametrize("T,d", [(0, 64), (1, 64), (4, 256), (300, 7168), (16384, 7168), (70000, 64), (5, 32768)])
def test_norm_grad_workspace_size(L, T, d):
    """At least one fp32 row, at most one for each of 296 CTAs, and never more than the rows."""
    n = moe.moe_rmsnorm_backward_workspace_size(T, d)
    assert n % 256 == 0 and n <= min(T, 296) * d * 4
    assert (n == 0) == (T == 0)
    assert T == 0 or n >= d * 4
    with pytest.raises(moe.MoEError):
        moe.moe_rmsnorm_backward_workspace_size(-1, d)


def test_quantize_int8_refusals(L):
    f = L.moe_quantize_int8_rows
    assert f(P, 0, 64, P, P, None) == 0
    assert f(P, -1, 64, P, P, None) == -1
    assert f(P, 4, 0, P, P, None) == -1
    assert f(P, 4, 32832, P, P, None) == -1
    assert f(P, 4, 96, P, P, None) == -2
    assert f(None, 4, 64, P, P, None) == -1
    assert f(P, 4, 64, None, P, None) == -1
    assert f(P, 4, 64, P, None, None) == -1
    assert f(ODD, 4, 64, P, P, None) == -2
    assert f(P, 4, 64, ODD, P, None) == -2


def _gemm(L, **kw):
    a = dict(xq=P, sx=P, Wq=P, sw=P, T=4, K=128, N=128, out=P, ws=P, ws_bytes=256)
    a.update(kw)
    return L.moe_gemm_int8(*[a[n] for n in ("xq", "sx", "Wq", "sw", "T", "K", "N", "out", "ws", "ws_bytes")], None)


def _grouped(L, **kw):
    a = dict(xq=P, sx=P, counts=P, offsets=P, Wq=P, sw=P, T=4, K=128, N=128, E=8, k=2, out=P, ws=P, ws_bytes=256)
    a.update(kw)
    return L.moe_grouped_gemm_int8(*[a[n] for n in ("xq", "sx", "counts", "offsets", "Wq", "sw", "T", "K", "N", "E",
                                                    "k", "out", "ws", "ws_bytes")], None)


@pytest.mark.parametrize("call", [_gemm, _grouped])
def test_int8_refusals(L, call):
    assert call(L, T=0) == 0
    assert call(L, T=-1) == -1
    assert call(L, T=1 << 31) == -1
    assert call(L, K=0) == -1
    assert call(L, N=0) == -1
    assert call(L, K=65536 + 64) == -1
    assert call(L, K=96) == -2
    assert call(L, N=96) == -2
    for name in ("xq", "sx", "Wq", "sw", "out", "ws"):
        assert call(L, **{name: None}) == -1, name
        assert call(L, **{name: ODD}) == -2, name
    assert call(L, ws_bytes=255) == -3


def test_grouped_int8_refusals(L):
    assert _grouped(L, counts=None) == -1
    assert _grouped(L, offsets=None) == -1
    assert _grouped(L, E=513) == -1
    assert _grouped(L, k=9, E=16) == -1
    assert _grouped(L, k=3, E=2) == -1
    assert _grouped(L, E=512, N=1 << 22) == -1               # E * N rows of weights past 2^31


def _permute(L, **kw):
    a = dict(idx=P, xq=P, sx=P, T=4, d=128, E=8, k=2, counts=P, offsets=P, perm=P, inv=P, xpq=P, sxp=P, ws=P,
             ws_bytes=1 << 30)
    a.update(kw)
    return L.moe_permute_int8(*[a[n] for n in ("idx", "xq", "sx", "T", "d", "E", "k", "counts", "offsets", "perm",
                                               "inv", "xpq", "sxp", "ws", "ws_bytes")], None)


def test_permute_int8_refusals(L):
    assert _permute(L, T=0) == 0
    assert _permute(L, T=-1) == -1
    assert _permute(L, d=96) == -2
    assert _permute(L, k=9, E=16) == -1
    assert _permute(L, E=513) == -1
    for name in ("idx", "xq", "sx", "counts", "offsets", "perm", "inv", "xpq", "sxp", "ws"):
        assert _permute(L, **{name: None}) == -1, name
    for name in ("xq", "xpq", "ws"):
        assert _permute(L, **{name: ODD}) == -2, name
    assert _permute(L, ws_bytes=1024) == -3


def test_sorted_rows_refusals(L):
    back = lambda y=P, inv=P, w=P, sh=None, T=4, k=2, d=128, out=P: L.moe_combine_weighted(y, inv, w, sh, T, k, d,
                                                                                           out, None)
    grad = lambda g=P, y=P, inv=P, w=P, T=4, k=2, d=128, dy=P, dw=P: L.moe_combine_weighted_backward(g, y, inv, w, T,
                                                                                                     k, d, dy, dw, None)
    sort = lambda g=P, inv=P, add=None, T=4, k=2, d=128, dx=P: L.moe_permute_backward(g, inv, add, T, k, d, dx, None)
    for f in (back, grad, sort):
        assert f(T=0) == 0
        assert f(T=-1) == -1
        assert f(k=0) == -1 and f(k=9) == -1
        assert f(d=0) == -1 and f(d=96) == -2
        assert f(T=1 << 30, k=2) == -1
        assert f(inv=None) == -1
    assert back(y=None) == -1 and back(w=None) == -1 and back(out=None) == -1
    assert back(y=ODD) == -2 and back(out=ODD) == -2 and back(sh=ODD) == -2
    assert grad(g=None) == -1 and grad(y=None) == -1 and grad(w=None) == -1 and grad(dy=None) == -1 and grad(dw=None) == -1
    assert grad(g=ODD) == -2 and grad(y=ODD) == -2 and grad(dy=ODD) == -2
    assert sort(g=None) == -1 and sort(dx=None) == -1 and sort(add=ODD) == -2 and sort(g=ODD) == -2


# ---------------------------------------------------------------- the definitions themselves

def test_norm_gradient_formula_against_autograd_and_differences():
    g = R.gen(1)
    s = torch.randn(3, 64, generator=g, dtype=R.D, requires_grad=True)
    w = torch.randn(64, generator=g, dtype=R.D, requires_grad=True)
    dy = torch.randn(3, 64, generator=g, dtype=R.D)
    eps = 1e-3
    y = R.rmsnorm(s, w, eps)
    gs, gw = torch.autograd.grad(y, (s, w), dy)
    dx, dw, _, _ = R.rmsnorm_grad(dy, s.detach(), w.detach(), eps)
    assert torch.allclose(dx, gs, rtol=1e-12, atol=1e-13) and torch.allclose(dw, gw, rtol=1e-12, atol=1e-13)
    h = 1e-6
    for r, c in ((0, 0), (1, 17), (2, 63)):
        e = torch.zeros_like(s)
        e[r, c] = h
        diff = ((R.rmsnorm(s.detach() + e, w.detach(), eps) - R.rmsnorm(s.detach() - e, w.detach(), eps)) * dy).sum() / (2 * h)
        assert abs(float(diff - dx[r, c])) < 1e-8


def test_return_gradient_formula_against_autograd():
    g = R.gen(2)
    T, k, d, E = 5, 3, 64, 4
    idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
    idx[2, 1] = E + 3                                        # a dropped pair
    _, _, _, inv = R.permutation(idx, E)
    y = torch.randn(T * k, d, generator=g, dtype=R.D, requires_grad=True)
    w = torch.rand(T, k, generator=g, dtype=R.D, requires_grad=True)
    dout = torch.randn(T, d, generator=g, dtype=R.D)
    out, _ = R.combine(y, inv, w)
    gy, gw = torch.autograd.grad(out, (y, w), dout)
    dy, dw, _ = R.combine_grad(dout, y.detach(), inv, w.detach())
    assert torch.allclose(gw, dw, rtol=1e-12, atol=1e-13)
    for q, pos in enumerate(inv.tolist()):
        if pos >= 0:
            assert torch.allclose(gy[pos], dy[q], rtol=1e-12, atol=1e-13)
    assert float(dw[2, 1]) == 0.0


def test_int8_scale_rule():
    y = torch.tensor([[127.0, -127.0, 63.5, 0.0], [0.0, 0.0, 0.0, 0.0], [1.0, -0.5, 0.25, 2.0 ** -20]])
    v, scale = R.int8_rows(y)
    assert scale.tolist() == [1.0, 1.0, 1.0 / 127]
    assert torch.round(v).tolist() == [[127, -127, 64, 0], [0, 0, 0, 0], [127, -64, 32, 0]]


# ---------------------------------------------------------------- how a dense int8 product is cut

@pytest.fixture(scope="module")
def shape_of(tmp_path_factory):
    here = os.path.dirname(os.path.abspath(__file__))
    out = str(tmp_path_factory.mktemp("shape") / "libshape.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-o", out,
                    os.path.join(here, "int8_shape_harness.cpp")], check=True)
    lib = C.CDLL(out)
    i64 = C.c_int64
    lib.int8_shape_of.argtypes = [i64, i64, i64, C.c_int, C.c_int, C.POINTER(C.c_int), C.c_int, C.POINTER(i64)]
    lib.int8_grouped_pair_of.argtypes = [i64, i64, i64, i64, C.c_int, C.c_int, C.c_int]

    def f(T, K, N, sms=148, can_pair=True, pairs=-1, clusters=B200_CLUSTERS):
        buf = (i64 * 5)()
        lib.int8_shape_of(T, K, N, sms, int(can_pair), (C.c_int * 9)(*clusters), pairs, buf)
        return tuple(buf)
    f.grouped = lib.int8_grouped_pair_of
    return f


SINGLE, PAIR, SPLIT = 0, 1, 2
B200_CLUSTERS = (0, 148, 74, 45, 33, 26, 22, 15, 15)       # of 0..8 CTAs that fit a B200 at once


@pytest.mark.parametrize("sms,can_pair,pairs,clusters", [
    (148, True, -1, B200_CLUSTERS), (148, True, 0, B200_CLUSTERS), (148, True, 1, B200_CLUSTERS),
    (148, False, 1, B200_CLUSTERS), (148, False, -1, (0,) * 9), (1, True, -1, (0,) * 9), (7, False, -1, (0, 7, 3, 2, 1, 1, 1, 1, 0))])
def test_int8_cut_covers_the_product(shape_of, sms, can_pair, pairs, clusters):
    """Every cut: the units cover the rows, tiles fit the accumulator and the form's alignment, and CTAs that share a
    tile have a K block each and are all resident at once."""
    for T in (1, 2, 15, 16, 17, 33, 100, 255, 256, 257, 1000, 4096, 16385, 1 << 20):
        for K in (64, 128, 192, 1024, 7168, 65536):
            for N in (64, 128, 192, 2048, 7168, 65536):
                form, chunk, units, split, tiles = shape_of(T, K, N, sms, can_pair, pairs, clusters)
                what = (T, K, N, form, chunk, units, split, tiles)
                assert form in (SINGLE, PAIR, SPLIT), what
                assert chunk % (32 if form == PAIR else 16) == 0 and 16 <= chunk <= 256, what
                assert (units - 1) * chunk < T <= units * chunk, what
                rows = 256 if form == PAIR else 128
                assert tiles == -(-N // rows) * units, what
                if form == SPLIT:
                    assert 2 <= split <= 8 and split <= -(-K // 128) and tiles <= clusters[split], what
                else:
                    assert split == 1, what
                if pairs == 1 and can_pair:
                    assert form == PAIR, what
                if pairs == 0 or not can_pair:
                    assert form != PAIR, what


def test_int8_cut_reaches_every_form(shape_of):
    forms = {shape_of(T, K, N)[0] for T, K, N in ((8, 1024, 2048), (8, 7168, 4096), (8192, 7168, 4096))}
    assert forms == {SINGLE, PAIR, SPLIT}
    assert [shape_of(1, K, N)[3] for K, N in ((7168, 7168), (7168, 4096), (16384, 512))] == [2, 4, 8]
    # rows of a tile shrink until the SMs are busy
    assert shape_of(256, 1024, 2048)[1] < 256 and shape_of(8192, 1024, 2048)[1] >= 192
    # more tiles than a launch counts are refused (units 0), not wrapped
    assert shape_of((1 << 31) - 1, 64, (1 << 31) - 64)[2] == 0


def test_grouped_int8_takes_pairs_for_wide_segments(shape_of):
    g = shape_of.grouped
    assert g(4096 * 8, 2048, 2048, 64, 148, 1, -1) == 1
    assert g(32 * 8, 2048, 2048, 64, 148, 1, -1) == 0
    assert g(4096 * 8, 2048, 2048, 64, 148, 0, -1) == 0 and g(4096 * 8, 2048, 2048, 64, 148, 0, 1) == 0
    assert g(1, 64, 64, 1, 148, 1, 1) == 1 and g(1 << 20, 2048, 2048, 8, 148, 1, 0) == 0
