"""The int8 product's forms beside each other, and segments that a grouped product refuses (marked gpu)."""

from __future__ import annotations

import pytest
import torch

from grouped_gemm_02_b200 import moe
from tests import ops_helpers as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("counts,offsets", [([10, 9], [0, 3, 16]), ([16, 1], [0, 0, 16]), ([6, 6, 6], [0, 5, 10, 16])])
def test_grouped_gemm_int8_refuses_segments_that_overlap(counts, offsets):
    """Each segment inside the rows, more rows in all than there are: an error bit, and nothing is written."""
    T, k, K, N, E = 8, 2, 128, 128, len(counts)
    xq, sx = R.codes(1, T * k, K).to(DEV), R.scales(2, T * k).to(DEV)
    wq, sw = R.codes(3, E, N, K).to(DEV), R.scales(4, E, N).to(DEV)
    ws = moe.new_workspace(T, 64, 64, E, k)
    out = torch.full((T * k, N), 7.0, dtype=torch.bfloat16, device=DEV)
    t = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
    moe.moe_grouped_gemm_int8(xq, sx, t(counts), t(offsets), wq, sw, T, k, ws, out=out)
    assert moe.moe_get_device_error(ws) == moe.DEVERR_PLAN
    assert (out == 7.0).all()
