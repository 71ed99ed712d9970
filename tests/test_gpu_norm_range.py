"""The norm where its squares leave fp32, and where products on the way to an ordinary result do (marked gpu).

Tolerances as in the ordinary range: one rounding to bf16 and 2^-17 for the fp32 steps before it."""

from __future__ import annotations

import pytest
import torch

from grouped_gemm_02_b200 import moe
from tests import ops_helpers as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
NORM32 = 2.0 ** -17


def _rows(d, sizes, seed):
    """One row for each size, its largest values a few times that; the last has a single large value."""
    x = torch.randn(len(sizes) + 1, d, generator=R.gen(seed), dtype=torch.float64).clamp(-3, 3)
    x[:-1] *= torch.tensor(sizes, dtype=torch.float64)[:, None]
    x[-1, d // 2] = -3.3e38
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("d", [64, 1088, 7168, 32768])
def test_rmsnorm_of_rows_whose_squares_leave_fp32(d):
    x = _rows(d, [1e18, 1e19, 1e20, 1e37, 1e38, 1.0, 1e-25, 1e-38], seed=1)
    w = (1 + 0.3 * torch.randn(d, generator=R.gen(2))).to(torch.bfloat16)
    ref = R.rmsnorm(x, w, 1e-6)
    y = moe.moe_rmsnorm(x.to(DEV), w.to(DEV), 1e-6)
    R.within(y, ref, (R.BF16 + NORM32) * ref.abs() + R.TINY, f"d={d}")
    q, sc = moe.moe_rmsnorm_int8(x.to(DEV), w.to(DEV), 1e-6)
    rq, rs = moe.moe_quantize_int8_rows(y)
    assert torch.equal(q, rq) and torch.equal(sc, rs)
    if d % 128 == 0:
        q, sc = moe.moe_rmsnorm_fp8(x.to(DEV), w.to(DEV), 1e-6)
        rq, rs = moe.moe_quantize_fp8_rows(y)
        assert torch.equal(q, rq) and torch.equal(sc, rs)


def test_rmsnorm_of_many_large_rows():
    """From two rows an SM on, where a thread holds twice as much of a row; and with a residual."""
    T, d = 400, 1088
    x = _rows(d, [10.0 ** (37 * t / T) for t in range(T - 1)], seed=3)
    r = _rows(d, [10.0 ** (18 + 19 * t / T) for t in range(T - 1)], seed=4)
    r[-1] = 0
    w = (1 + 0.3 * torch.randn(d, generator=R.gen(5))).to(torch.bfloat16)
    y, s = moe.moe_rmsnorm(x.to(DEV), w.to(DEV), 1e-6, residual=r.to(DEV))
    assert torch.equal(s.cpu(), R.add_bf16(x, r))
    ref = R.rmsnorm(s, w.to(DEV), 1e-6)
    R.within(y, ref, (R.BF16 + NORM32) * ref.abs() + R.TINY, "with a residual")


@pytest.mark.parametrize("eps", [1e-30, 1e-38, 2e-44])
def test_rmsnorm_of_small_rows_and_a_small_eps(eps):
    d = 448
    eps = float(torch.tensor(eps, dtype=torch.float32))          # the value the call gets
    x = _rows(d, [1.0, 1e-12, 1e-15, 1e-18, 1e-19, 1e-20, 1e-21, 1e-22, 1e-23, 1e-30, 0.0], seed=6)
    w = (1 + 0.3 * torch.randn(d, generator=R.gen(7))).to(torch.bfloat16)
    ref = R.rmsnorm(x, w, eps)
    y = moe.moe_rmsnorm(x.to(DEV), w.to(DEV), eps)
    R.within(y, ref, (R.BF16 + NORM32) * ref.abs() + R.TINY, f"eps={eps}")


@pytest.mark.parametrize("size,weight", [(1e10, 1e30), (1e30, 1e12), (1e38, 1e37), (1e-20, 1e-22), (1e-10, 1e-36)])
def test_rmsnorm_whose_stream_times_weight_leaves_fp32(size, weight):
    """s * w alone is beyond fp32 or below its normal numbers, s / rms * w is not."""
    d = 1152
    x = _rows(d, [size, size / 8], seed=8)
    w = (weight * (1 + 0.3 * torch.randn(d, generator=R.gen(9), dtype=torch.float64))).to(torch.bfloat16)
    ref = R.rmsnorm(x, w, 1e-38)
    assert ref.abs().max() < 3.3e38
    y = moe.moe_rmsnorm(x.to(DEV), w.to(DEV), 1e-38)
    R.within(y, ref, (R.BF16 + NORM32) * ref.abs() + R.TINY, f"size={size} weight={weight}")


@pytest.mark.parametrize("eps", [1e-6, 1e-44])
@pytest.mark.parametrize("d", [64, 7168])
def test_rmsnorm_of_non_finite_rows(d, eps):
    """NaN of either sign, infinities of either sign and both together, beside rows that are finite."""
    x = _rows(d, [1.0, 1.0, 1e20, 1.0, 1.0], seed=10)
    x.view(torch.int16)[0, 3] = -64                              # 0xFFC0, a negative NaN
    x[1, 5], x[2, 6], x[3, 7], x[3, 8] = float("nan"), float("-inf"), float("inf"), float("-inf")
    w = (1 + 0.3 * torch.randn(d, generator=R.gen(11))).to(torch.bfloat16)
    y = moe.moe_rmsnorm(x.to(DEV), w.to(DEV), eps).cpu()
    ref = R.rmsnorm(x, w, eps)
    assert torch.equal(torch.isnan(y), torch.isnan(ref))
    R.within(y, ref, (R.BF16 + NORM32) * ref.abs() + R.TINY, f"d={d}")
    _, sc = moe.moe_rmsnorm_int8(x.to(DEV), w.to(DEV), eps)
    assert torch.isnan(sc.cpu()).tolist() == [True] * 4 + [False] * 2


# ---------------------------------------------------------------- gradient

def _check_grad(dy, s, w, eps, ds, what):
    """As in the ordinary range; a dx beyond the largest bf16 by half a step or more is infinite."""
    dx, dw = moe.moe_rmsnorm_backward(dy.to(DEV), s.to(DEV), w.to(DEV), eps, dxsum=None if ds is None else ds.to(DEV))
    rx, rw, mx, mw = R.rmsnorm_grad(dy, s, w, eps, ds)
    rx = torch.where(rx.abs() >= 2.0 ** 128 * (1 - 2.0 ** -9), torch.copysign(torch.full_like(rx, float("inf")), rx), rx)
    R.within(dx, rx, R.BF16 * rx.abs() + NORM32 * mx + R.TINY, f"dx {what}")
    steps = -(-s.shape[0] // 296) + 8 + 296 + 8
    R.within(dw, rw, (NORM32 + steps * R.F32) * mw + R.TINY, f"dweight {what}")


@pytest.mark.parametrize("with_stream", [False, True])
@pytest.mark.parametrize("d", [64, 1088, 7168, 8256, 32768])
def test_rmsnorm_backward_of_rows_whose_squares_leave_fp32(d, with_stream):
    s = _rows(d, [1.0, 1e18, 1e19, 1e20, 2.0, 1e30, 1e37, 1e-25, 3.0], seed=20)
    s[-1, d // 2] = 3e24
    w = (1 + 0.3 * torch.randn(d, generator=R.gen(21))).to(torch.bfloat16)
    dy = R.randn(22, *s.shape, std=0.1)
    ds = R.randn(23, *s.shape, std=1e-22) if with_stream else None
    _check_grad(dy, s, w, 1e-6, ds, f"d={d}")


@pytest.mark.parametrize("eps", [1e-30, 1e-38, 2e-44])
def test_rmsnorm_backward_of_small_rows_and_a_small_eps(eps):
    d = 448
    eps = float(torch.tensor(eps, dtype=torch.float32))
    s = _rows(d, [1.0, 1e-12, 1e-15, 1e-18, 1e-19, 1e-20, 1e-21, 1e-22, 1e-23, 1e-30], seed=24)[:-1]
    w = (1 + 0.3 * torch.randn(d, generator=R.gen(25))).to(torch.bfloat16)
    _check_grad(R.randn(26, *s.shape, std=1e-4), s, w, eps, None, f"eps={eps}")


@pytest.mark.parametrize("size,grad,weight", [(1e10, 1e22, 1e10), (1e19, 1e20, 1.0), (1e-3, 1e25, 1e12)])
def test_rmsnorm_backward_whose_products_leave_fp32(size, grad, weight):
    """dy * weight is within fp32, its products with the stream are not."""
    d = 1152
    s = _rows(d, [size, size / 4, 4 * size], seed=27)[:-1]
    w = (weight * (1 + 0.3 * torch.randn(d, generator=R.gen(28)))).to(torch.bfloat16)
    dy = (grad * torch.randn(3, d, generator=R.gen(29))).to(torch.bfloat16)
    _check_grad(dy, s, w, 1e-12, None, f"size={size}")


@pytest.mark.parametrize("T,d", [(5, 64), (5, 7168), (700, 448)])
def test_rmsnorm_backward_of_non_finite_rows(T, d):
    """A NaN or an infinity stays in its row of dx; of dweight a NaN row takes every column, an infinity its own."""
    w = (1 + 0.3 * torch.randn(d, generator=R.gen(30))).to(torch.bfloat16)
    dy = R.randn(31, T, d, std=0.1)
    for value, columns in ((float("nan"), d), (float("inf"), 1), (float("-inf"), 1)):
        s = _rows(d, [1.0] * (T - 1), seed=32)
        s[-1] = 1
        s[2, 9] = value
        dx, dw = moe.moe_rmsnorm_backward(dy.to(DEV), s.to(DEV), w.to(DEV), 1e-6)
        rx, rw, mx, mw = R.rmsnorm_grad(dy, s, w, 1e-6)
        assert torch.equal(torch.isnan(dx.cpu()), torch.isnan(rx)) and int(torch.isnan(dx).sum()) == d
        assert torch.equal(torch.isnan(dw.cpu()), torch.isnan(rw)) and int(torch.isnan(dw).sum()) == columns
        keep = torch.arange(T) != 2
        R.within(dx.cpu()[keep], rx[keep], (R.BF16 * rx.abs() + NORM32 * mx + R.TINY)[keep], "rows beside")
