"""Residual addition with root-mean-square norm, its gradient and the int8 row quantiser on the GPU against
their 64-bit definitions (marked gpu).

Tolerances, each result rounded to bf16 once (half a step, 2^-8 relative).  Before that, fp32: in the gradient the
mean of squares adds at most 8 * 4 values a thread and 10 levels of a tree, so its relative error is below 64 * 2^-24;
rsqrt halves it and adds 2 ulp, and two products follow: below 2^-18 in all, written as 2^-17.  The forward pass
stays within that too."""

from __future__ import annotations

import pytest
import torch

from grouped_gemm_02_b200 import moe
from tests import ops_helpers as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-5
NORM32 = 2.0 ** -17


def _rows(T, d, seed, std=1.0):
    """Rows of the residual stream: a few channels far larger than the rest, rows of very different size."""
    gamma = torch.exp(0.7 * torch.randn(d, generator=R.gen(seed + 1000)))
    size = torch.logspace(-3, 3, T)[:, None] if T > 1 else torch.ones(1, 1)
    return (torch.randn(T, d, generator=R.gen(seed)) * gamma * size * std).to(torch.bfloat16)


def _weight(d, seed):
    return (1 + 0.3 * torch.randn(d, generator=R.gen(seed))).to(torch.bfloat16)


SIZES = [(1, 64), (3, 192), (2, 256), (17, 1088), (5, 4096), (1, 7168), (297, 7168), (300, 64), (4, 8256), (3, 16384),
         (2, 32768), (700, 448)]


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("with_residual", [False, True])
def test_rmsnorm(T, d, with_residual):
    x, w = _rows(T, d, 1), _weight(d, 2)
    r = _rows(T, d, 3, std=2.0) if with_residual else None
    got = moe.moe_rmsnorm(x.to(DEV), w.to(DEV), EPS, residual=None if r is None else r.to(DEV))
    s = x
    if with_residual:
        got, xsum = got
        s = R.add_bf16(x, r)
        assert torch.equal(xsum.cpu(), s)
    ref = R.rmsnorm(s, w, EPS)
    R.within(got, ref, (R.BF16 + NORM32) * ref.abs() + R.TINY, f"rmsnorm T={T} d={d}")


def test_rmsnorm_zero_and_non_finite_rows():
    T, d = 5, 448
    x, w = _rows(T, d, 4), _weight(d, 5)
    x[0] = 0.0                       # stays zero: 1 / sqrt(eps) times 0
    x[2, 7] = float("nan")           # the row is NaN, its neighbours are not
    x[3, 9] = float("inf")           # mean of squares infinite: finite elements give 0, the infinite one NaN
    y = moe.moe_rmsnorm(x.to(DEV), w.to(DEV), EPS).cpu()
    assert (y[0] == 0).all()
    assert torch.isnan(y[2]).all()
    assert torch.isnan(y[3, 9]) and (y[3, torch.arange(d) != 9] == 0).all()
    ref = R.rmsnorm(x[[1, 4]], w, EPS)
    R.within(y[[1, 4]], ref, (R.BF16 + NORM32) * ref.abs(), "rows beside")
    q, sc = moe.moe_rmsnorm_int8(x.to(DEV), w.to(DEV), EPS)
    assert torch.isnan(sc[2]) and torch.isnan(sc[3]) and float(sc[0]) == 1.0 and (q[0] == 0).all()
    assert torch.isfinite(sc[[1, 4]]).all()


@pytest.mark.parametrize("T,d", [s for s in SIZES if s[1] % 128 == 0])
@pytest.mark.parametrize("with_residual", [False, True])
def test_rmsnorm_fp8_is_the_quantised_norm(T, d, with_residual):
    """Codes and scales are those of moe_quantize_fp8_rows (pinned to the oracle bit for bit) of moe_rmsnorm's y."""
    x, w = _rows(T, d, 6).to(DEV), _weight(d, 7).to(DEV)
    if T > 2:
        x[1, :128] = 0.0
    r = _rows(T, d, 8).to(DEV) if with_residual else None
    y = moe.moe_rmsnorm(x, w, EPS, residual=r)
    y, s = y if with_residual else (y, None)
    y2 = torch.empty_like(y)
    q, sc, *xsum = moe.moe_rmsnorm_fp8(x, w, EPS, residual=r, y=y2)
    rq, rs = moe.moe_quantize_fp8_rows(y)
    assert torch.equal(q, rq) and torch.equal(sc, rs) and torch.equal(y, y2)
    if with_residual:
        assert torch.equal(xsum[0], s)


def test_rmsnorm_fp8_blocks_at_the_edges():
    """Block maxima around 1.75 times a power of two, subnormal and non-finite values: the quantiser's codes and
    scales.  A weight of ones and one row size leave y = x / rms, so the blocks' values are set by the weight."""
    d = 2048
    x = torch.ones(4, d, dtype=torch.bfloat16)
    w = torch.ones(d)
    top = [448.0, 449.0, 450.0, 447.0, 1.75, 1.7578125, 3.5, 2.0 ** -120, 2.0 ** -126, 2.0 ** -130, 3e38, 0.0, 1.0]
    for b, v in enumerate(top):
        w[128 * b:128 * (b + 1)] = torch.linspace(-1, 1, 128) * v
    w[128 * 13 + 5], w[128 * 14 + 7], w[128 * 15 + 9] = float("nan"), float("inf"), float("-inf")
    w = w.to(torch.bfloat16).to(DEV)
    y = moe.moe_rmsnorm(x.to(DEV), w, 1e-30)
    q, sc = moe.moe_rmsnorm_fp8(x.to(DEV), w, 1e-30)
    rq, rs = moe.moe_quantize_fp8_rows(y)
    assert torch.equal(sc, rs) and torch.equal(q, rq)


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("with_residual", [False, True])
def test_rmsnorm_int8_is_the_quantised_norm(T, d, with_residual):
    x, w = _rows(T, d, 9).to(DEV), _weight(d, 10).to(DEV)
    r = _rows(T, d, 11).to(DEV) if with_residual else None
    y = moe.moe_rmsnorm(x, w, EPS, residual=r)
    y, s = y if with_residual else (y, None)
    y2 = torch.empty_like(y)
    q, sc, *xsum = moe.moe_rmsnorm_int8(x, w, EPS, residual=r, y=y2)
    rq, rs = moe.moe_quantize_int8_rows(y)
    assert torch.equal(q, rq) and torch.equal(sc, rs) and torch.equal(y, y2)
    if with_residual:
        assert torch.equal(xsum[0], s)


@pytest.mark.parametrize("T,d", SIZES)
def test_quantize_int8_rows(T, d):
    """scale: one fp32 division (2^-24).  code: v * (127 / amax) carries 2 roundings of a value up to 127."""
    x = _rows(T, d, 12)
    if T > 2:
        x[1] = 0.0
        x[2] *= 2.0 ** -110
    q, sc = moe.moe_quantize_int8_rows(x.to(DEV))
    keep = x.float().abs().amax(1) >= 2.0 ** -100              # a smaller row counts as zero
    assert (q.cpu()[~keep] == 0).all() and (sc.cpu()[~keep] == 1.0).all()
    v, scale = R.int8_rows(x[keep])
    R.within(sc.cpu()[keep], scale, R.F32 * scale, "scale")
    R.within(q.cpu()[keep], v, torch.full_like(v, 0.5 + 127 * 2 * R.F32), "codes")
    assert int(q.cpu()[keep].abs().max()) == 127


def test_quantize_int8_keeps_non_finite_rows_visible():
    x = _rows(6, 256, 13)
    x[0, 3], x[2, 255], x[4, 0] = float("nan"), float("inf"), float("-inf")
    q, sc = moe.moe_quantize_int8_rows(x.to(DEV))
    assert torch.isnan(sc.cpu()).tolist() == [True, False, True, False, True, False]
    big = torch.full((2, 64), 3.38e38).to(torch.bfloat16)
    q, sc = moe.moe_quantize_int8_rows(big.to(DEV))
    assert (q == 127).all() and torch.isfinite(sc).all()
    E = moe.moe_quantize_int8_rows(_rows(6, 256, 14).view(2, 3, 256).to(DEV))
    assert E[0].shape == (2, 3, 256) and E[1].shape == (2, 3)


# ---------------------------------------------------------------- gradient

@pytest.mark.parametrize("T,d", [(1, 64), (3, 192), (17, 1088), (5, 4096), (1, 7168), (600, 1024), (297, 7168),
                                 (3000, 64), (4, 8256), (3, 16384), (2, 16448), (2, 32768)])
@pytest.mark.parametrize("with_stream", [False, True])
def test_rmsnorm_backward(T, d, with_stream):
    """dx: the norm's fp32 error on every magnitude it adds.  dweight: a column adds at most ceil(T / 296) + 8 rows in
    a thread and its partials in at most 296 * 8 / 8 + 8 steps; each n carries the norm's error."""
    s, w, dy = _rows(T, d, 20), _weight(d, 21), R.randn(22, T, d, std=0.1)
    ds = R.randn(23, T, d, std=0.1) if with_stream else None
    dx, dw = moe.moe_rmsnorm_backward(dy.to(DEV), s.to(DEV), w.to(DEV), EPS,
                                      dxsum=None if ds is None else ds.to(DEV))
    rx, rw, mx, mw = R.rmsnorm_grad(dy, s, w, EPS, ds)
    R.within(dx, rx, R.BF16 * rx.abs() + NORM32 * mx + R.TINY, f"dx T={T} d={d}")
    steps = -(-T // 296) + 8 + 296 + 8
    R.within(dw, rw, (NORM32 + steps * R.F32) * mw + R.TINY, f"dweight T={T} d={d}")
    assert dw.dtype == torch.float32


def test_rmsnorm_backward_of_no_rows_and_reruns():
    d = 192
    e = torch.empty(0, d, dtype=torch.bfloat16, device=DEV)
    w = _weight(d, 24).to(DEV)
    dx, dw = moe.moe_rmsnorm_backward(e, e, w, EPS, dweight=torch.full((d,), 7.0, device=DEV))
    assert dx.shape == (0, d) and (dw == 0).all()
    assert moe.moe_rmsnorm(e, w, EPS).shape == (0, d)
    s, dy = _rows(999, d, 25).to(DEV), R.randn(26, 999, d).to(DEV)
    a, b = (moe.moe_rmsnorm_backward(dy, s, w, EPS) for _ in range(2))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_norm_past_32_bit_offsets():
    """Rows whose offsets pass 2^31 elements: the last rows, where an overflow would show."""
    T, d = 300_100, 7168                                    # 2.15e9 elements
    x = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
    part = _rows(100, d, 50).to(DEV)
    x[-100:] = part
    x[:-100] = 1.0
    w = _weight(d, 51).to(DEV)
    q, sc = moe.moe_rmsnorm_int8(x, w, EPS)
    q1, sc1 = moe.moe_rmsnorm_int8(part, w, EPS)
    assert torch.equal(q[-100:], q1) and torch.equal(sc[-100:], sc1)
    del q
    dy = torch.zeros_like(x)
    dy[-100:] = R.randn(52, 100, d).to(DEV)
    dx, dw = moe.moe_rmsnorm_backward(dy, x, w, EPS)
    rx, rw, mx, mw = R.rmsnorm_grad(dy[-100:], part, w, EPS)
    R.within(dx[-100:], rx, R.BF16 * rx.abs() + NORM32 * mx + R.TINY, "dx")
    R.within(dw, rw, (NORM32 + 400 * R.F32) * mw + R.TINY, "dweight")
    assert (dx[:-100] == 0).all()


def test_norm_in_place():
    """The buffers that the documentation allows to coincide."""
    T, d = 33, 1088
    x, r, w = _rows(T, d, 27).to(DEV), _rows(T, d, 28).to(DEV), _weight(d, 29).to(DEV)
    y, s = moe.moe_rmsnorm(x, w, EPS, residual=r)
    r1 = r.clone()
    y1, s1 = moe.moe_rmsnorm(x, w, EPS, residual=r1, xsum=r1)
    assert s1 is r1 and torch.equal(r1, s) and torch.equal(y1, y)
    x1, r1 = x.clone(), r.clone()
    y1, _ = moe.moe_rmsnorm(x1, w, EPS, residual=r1, xsum=r1, y=x1)
    assert torch.equal(x1, y) and torch.equal(r1, s)
    dy, ds = R.randn(30, T, d).to(DEV), R.randn(31, T, d).to(DEV)
    dx, dw = moe.moe_rmsnorm_backward(dy, s, w, EPS, dxsum=ds)
    for buf in ("dy", "ds"):
        a, b = dy.clone(), ds.clone()
        dx1, dw1 = moe.moe_rmsnorm_backward(a, s, w, EPS, dxsum=b, dx=a if buf == "dy" else b)
        assert torch.equal(dx1, dx) and torch.equal(dw1, dw)


@pytest.mark.parametrize("d", [128, 1152, 7168])
def test_norm_of_tensors_aligned_to_16_bytes_only(d):
    """The documented alignment is 16 bytes: views that start there give what aligned copies give."""
    T = 9
    def view(t):
        buf = torch.empty(t.numel() + 8, dtype=t.dtype, device=DEV)[8:].view(t.shape)
        assert buf.data_ptr() % 32 == 16
        return buf.copy_(t)
    x, r, w = _rows(T, d, 40), _rows(T, d, 41), _weight(d, 42)
    y, s = moe.moe_rmsnorm(x.to(DEV), w.to(DEV), EPS, residual=r.to(DEV))
    ov = view(torch.zeros(T, d, dtype=torch.bfloat16))
    y1, s1 = moe.moe_rmsnorm(view(x), view(w), EPS, residual=view(r), xsum=ov)
    assert torch.equal(y, y1) and torch.equal(s, s1)
    for f in (moe.moe_rmsnorm_fp8, moe.moe_rmsnorm_int8):
        a = f(x.to(DEV), w.to(DEV), EPS, residual=r.to(DEV))
        b = f(view(x), view(w), EPS, residual=view(r), y=view(x))
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    q, sc = moe.moe_quantize_int8_rows(view(x))
    q1, sc1 = moe.moe_quantize_int8_rows(x.to(DEV))
    assert torch.equal(q, q1) and torch.equal(sc, sc1)
    dy, ds = R.randn(43, T, d), R.randn(44, T, d)
    g = moe.moe_rmsnorm_backward(dy.to(DEV), s, w.to(DEV), EPS, dxsum=ds.to(DEV))
    g1 = moe.moe_rmsnorm_backward(view(dy), view(s.cpu()), view(w), EPS, dxsum=view(ds), dx=view(dy))
    assert torch.equal(g[0], g1[0]) and torch.equal(g[1], g1[1])


def test_norm_refuses_what_it_cannot_take():
    x, w = _rows(4, 256, 32).to(DEV), _weight(256, 33).to(DEV)
    with pytest.raises(AssertionError, match="contiguous"):
        moe.moe_rmsnorm(x[:, ::2], w[::2], EPS)
    with pytest.raises(AssertionError, match="x: expected"):
        moe.moe_rmsnorm(x.float(), w, EPS)
    with pytest.raises(AssertionError, match="weight"):
        moe.moe_rmsnorm(x, w[:128], EPS)
    with pytest.raises(AssertionError, match="x: expected"):
        moe.moe_rmsnorm(x.cpu(), w, EPS)
    with pytest.raises(AssertionError, match="residual"):
        moe.moe_rmsnorm(x, w, EPS, xsum=x)
    with pytest.raises(moe.MoEError):
        moe.moe_rmsnorm(x, w, 0.0)
    with pytest.raises(moe.MoEError):
        moe.moe_rmsnorm_fp8(x[:, :192].contiguous(), w[:192].contiguous(), EPS)
    off = torch.empty(4 * 256 + 4, dtype=torch.bfloat16, device=DEV)[4:].view(4, 256)
    with pytest.raises(moe.MoEError, match="alignment"):
        moe.moe_rmsnorm(off, w, EPS)
