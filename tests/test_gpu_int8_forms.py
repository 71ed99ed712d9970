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


# Sizes whose K range a cluster shares (the cut itself is tested on the CPU), by rows a tile and CTAs a cluster:
# 16 x 6, 48 x 6, 96 x 2, 160 x 4, 96 x 8, 256 x 4.  The last rows are no multiple of 16.
SHARED_K = [(5, 4096, 2048), (90, 7168, 1088), (190, 7168, 4096), (150, 7168, 4096), (250, 32768, 448),
            (250, 16384, 4096)]


@pytest.mark.parametrize("T,K,N", SHARED_K)
def test_a_shared_k_range_gives_the_bits_of_the_other_forms(T, K, N):
    """Against CTA pairs, and against single CTAs and pairs of the grouped product with one expert."""
    xq, sx = R.codes(T, T, K).to(DEV), R.scales(T + 1, T).to(DEV)
    wq, sw = R.codes(T + 2, N, K).to(DEV), R.scales(T + 3, N, mean=0.001).to(DEV)
    ws = moe.new_workspace(T, 64, 64, 1, 1)
    got = moe.moe_gemm_int8(xq, sx, wq, sw, ws)
    t = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)
    try:
        for pairs in (0, 1):
            moe.moe_set_policy(moe.POLICY_CTA_PAIRS, pairs)
            one = moe.moe_grouped_gemm_int8(xq, sx, t(T), t(0, T), wq[None], sw[None], T, 1, ws)
            assert torch.equal(got, one), f"pairs={pairs}"
        assert torch.equal(got, moe.moe_gemm_int8(xq, sx, wq, sw, ws))
    finally:
        moe.moe_set_policy(moe.POLICY_CTA_PAIRS, -1)
    assert moe.moe_get_device_error(ws) == 0
    ref = R.int8_gemm(xq, sx, wq, sw)
    R.within(got, ref, (R.BF16 + 2.0 ** -21) * ref.abs() + R.TINY, f"T={T} K={K} N={N}")
