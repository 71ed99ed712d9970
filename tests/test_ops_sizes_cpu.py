"""Sizes that the norm's gradient refuses, asked of its workspace size first (CPU)."""

import pytest

from grouped_gemm_02_b200 import build, moe


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    moe.lib()


@pytest.mark.parametrize("d", [1, 4, 7, 8, 63, 65, 100, 32767])
@pytest.mark.parametrize("T", [0, 1, 5, 300])
def test_norm_grad_workspace_size_refuses_odd_rows(T, d):
    """The status that moe_rmsnorm_backward gives for such rows: a user meets the size function first."""
    with pytest.raises(moe.MoEError, match="alignment"):
        moe.moe_rmsnorm_backward_workspace_size(T, d)


@pytest.mark.parametrize("d", [0, -64, 32832, 1 << 40])
def test_norm_grad_workspace_size_refuses_sizes_out_of_range(d):
    with pytest.raises(moe.MoEError, match="invalid argument"):
        moe.moe_rmsnorm_backward_workspace_size(4, d)
