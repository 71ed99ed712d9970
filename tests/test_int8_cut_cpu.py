"""The sizes at which the GPU tests compare a shared K range with the other forms are cut that way (CPU)."""

import pytest

from tests.test_gpu_int8_forms import SHARED_K
from tests.test_ops_cpu import PAIR, SPLIT, shape_of  # noqa: F401

CUT = {(5, 4096, 2048): (16, 6), (90, 7168, 1088): (48, 6), (190, 7168, 4096): (96, 2), (150, 7168, 4096): (160, 4),
       (250, 32768, 448): (96, 8), (250, 16384, 4096): (256, 4)}


@pytest.mark.parametrize("T,K,N", SHARED_K)
def test_int8_sizes_that_share_a_k_range(shape_of, T, K, N):  # noqa: F811
    form, chunk, _, split, _ = shape_of(T, K, N)
    assert (form, (chunk, split)) == (SPLIT, CUT[T, K, N])
    assert shape_of(T, K, N, pairs=1)[0] == PAIR
    assert shape_of.grouped(T, K, N, 1, 148, 1, 0) == 0 and shape_of.grouped(T, K, N, 1, 148, 1, 1) == 1
