"""Buffers that the sorted-row entry points allow to coincide (marked gpu): the same bits as with buffers of their
own, at every instance of the kernels -- one to eight slots a token, short rows that share a CTA and long ones, few
tokens and many."""

from __future__ import annotations

import pytest
import torch

from grouped_gemm_02_b200 import moe
from grouped_gemm_02_b200 import workload as wl
from tests import ops_helpers as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _case(T, k, d, seed):
    idx = wl.random_routing(T, 9, k, 0.5, seed=seed)
    idx[T // 3, k - 1] = -1                                      # a dropped pair
    _, _, _, inv = R.permutation(idx, 9)
    return R.randn(seed, T * k, d).to(DEV), inv.to(DEV), wl.random_gates(T, k, seed).to(DEV), R.randn(seed + 1, T, d).to(DEV)


@pytest.mark.parametrize("k", [1, 2, 3, 8])
@pytest.mark.parametrize("T,d", [(5, 64), (333, 256), (301, 2112), (7, 16384)])
def test_return_into_the_rows_added(T, k, d):
    y, inv, w, add = _case(T, k, d, seed=31)
    for f in (lambda a, o: moe.moe_combine_weighted(y, inv, w, shared_out=a, out=o),
              lambda a, o: moe.moe_permute_backward(y, inv, T, k, addend=a, dx=o)):
        want = f(add, None)
        buf = add.clone()
        assert f(buf, buf) is buf and torch.equal(buf, want)


@pytest.mark.parametrize("k", [1, 3, 8])
@pytest.mark.parametrize("T,d", [(65, 320), (333, 128), (333, 512), (301, 7168)])
def test_return_gradient_into_the_rows(T, k, d):
    y, inv, w, dout = _case(T, k, d, seed=33)
    dy, dw = moe.moe_combine_weighted_backward(dout, y, inv, w)
    buf = y.clone()
    dy1, dw1 = moe.moe_combine_weighted_backward(dout, buf, inv, w, dy_p=buf)
    pos = inv[inv >= 0].long()
    assert dy1 is buf and torch.equal(buf[pos], dy[pos]) and torch.equal(dw1, dw)
