"""The int8 row quantiser on the GPU against its definition, at every mantissa of a row's largest magnitude
(marked gpu): v * 127 / max|v| is exact in 64 bits where it is a tie and far from one elsewhere, so the codes are
equal, not near."""

from __future__ import annotations

import pytest
import torch

from grouped_gemm_02_b200 import moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("exponent", [-90, 0, 100])
def test_codes_of_every_mantissa(exponent):
    top = torch.arange(128, 256, dtype=torch.float64)
    v = torch.cat([top * 2.0 ** -s for s in range(11)])
    v = torch.cat([v, -v])                                       # 2816 = 44 * 64 values a row
    rows = torch.where(v.abs()[None, :] <= top[:, None], v[None, :], torch.zeros(()).double())
    x = (rows * 2.0 ** exponent).to(torch.bfloat16)
    assert torch.equal(x.double(), rows * 2.0 ** exponent)
    q, sc = moe.moe_quantize_int8_rows(x.to(DEV))
    want = torch.round(rows * 127 / top[:, None])
    assert torch.equal(q.cpu().double(), want)
    assert (want.abs() == 64).any(1).all()                       # each row has its tie, 63.5
    unit = top * 2.0 ** exponent / 127
    assert ((sc.cpu().double() - unit).abs() <= 2.0 ** -24 * unit).all()
