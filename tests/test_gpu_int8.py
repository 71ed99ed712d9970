"""The int8 matrix product on the GPU, of one matrix and of one an expert, against 64-bit sums (marked gpu).

The integer sum is exact.  After it: one conversion to fp32, two products (3 * 2^-24) and one rounding to
bf16 (2^-8): tolerance (2^-8 + 2^-21) of the result."""

from __future__ import annotations

import pytest
import torch

from grouped_gemm_02_b200 import moe
from grouped_gemm_02_b200 import workload as wl
from tests import ops_helpers as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
REL = R.BF16 + 2.0 ** -21


def _ws(T, E=1, k=1):
    return moe.new_workspace(T, 64, 64, E, k)


def _dense(T, K, N, seed, lo=-127, hi=127):
    xq, wq = R.codes(seed, T, K, lo=lo, hi=hi), R.codes(seed + 1, N, K, lo=lo, hi=hi)
    return xq, R.scales(seed + 2, T), wq, R.scales(seed + 3, N, mean=0.001)


DENSE = [(1, 64, 64), (1, 7168, 2048), (2, 192, 448), (8, 7168, 4096), (16, 128, 128), (17, 4096, 1088),
         (33, 2048, 7168), (64, 1088, 192), (100, 320, 128), (255, 512, 704), (256, 16384, 256), (257, 640, 640),
         (300, 2048, 19200), (513, 1024, 2112), (1000, 2048, 1024), (2048, 704, 4096), (4100, 256, 2304)]


@pytest.mark.parametrize("T,K,N", DENSE)
def test_gemm_int8(T, K, N):
    xq, sx, wq, sw = _dense(T, K, N, seed=T + K)
    ws = _ws(T)
    out = torch.full((T + 3, N), 7.0, dtype=torch.bfloat16, device=DEV)     # rows behind the last stay as they are
    moe.moe_gemm_int8(xq.to(DEV), sx.to(DEV), wq.to(DEV), sw.to(DEV), ws, out=out[:T])
    assert moe.moe_get_device_error(ws) == 0
    ref = R.int8_gemm(xq.to(DEV), sx.to(DEV), wq.to(DEV), sw.to(DEV))
    R.within(out[:T], ref, REL * ref.abs() + R.TINY, f"T={T} K={K} N={N}")
    assert (out[T:] == 7.0).all()


@pytest.fixture
def pairs(request):
    moe.moe_set_policy(moe.POLICY_CTA_PAIRS, request.param)
    yield request.param
    moe.moe_set_policy(moe.POLICY_CTA_PAIRS, -1)


@pytest.mark.parametrize("pairs", [0, 1], indirect=True)
@pytest.mark.parametrize("T,K,N", [(1, 64, 64), (16, 128, 128), (17, 4096, 1088), (33, 2048, 320), (257, 640, 640),
                                   (1000, 2048, 1024), (300, 2048, 19200)])
def test_gemm_int8_every_form(pairs, T, K, N):
    """Integer sums: single CTAs, CTA pairs and shared K ranges give the same bits."""
    xq, sx, wq, sw = (t.to(DEV) for t in _dense(T, K, N, seed=T + N))
    got = moe.moe_gemm_int8(xq, sx, wq, sw, _ws(T))
    moe.moe_set_policy(moe.POLICY_CTA_PAIRS, -1)
    rule = moe.moe_gemm_int8(xq, sx, wq, sw, _ws(T))
    assert torch.equal(got, rule)
    ref = R.int8_gemm(xq, sx, wq, sw)
    R.within(got, ref, REL * ref.abs() + R.TINY, f"pairs={pairs} T={T} K={K} N={N}")


@pytest.mark.parametrize("T,K,N", [(1, 7168, 7168), (1, 7168, 4096), (3, 16384, 512)])
def test_gemm_int8_shared_k_ranges_rerun(T, K, N):
    """Two, four and eight CTAs a tile: the same bits in every run, and with no rows or channels lost."""
    xq, sx, wq, sw = (t.to(DEV) for t in _dense(T, K, N, seed=N))
    a, b = (moe.moe_gemm_int8(xq, sx, wq, sw, _ws(T)) for _ in range(2))
    assert torch.equal(a, b)
    ref = R.int8_gemm(xq, sx, wq, sw)
    R.within(a, ref, REL * ref.abs() + R.TINY, f"T={T} K={K} N={N}")


def test_gemm_int8_past_32_bit_offsets():
    """Codes and results whose offsets pass 2^31: the last rows, where an overflow would show."""
    T, K, N = 300_000, 64, 7232                         # T * N = 2.17e9 results
    xq, sx = R.codes(5, T, K).to(DEV), R.scales(6, T).to(DEV)
    wq, sw = R.codes(7, N, K).to(DEV), R.scales(8, N, mean=0.001).to(DEV)
    out = moe.moe_gemm_int8(xq, sx, wq, sw, _ws(1))
    for a in (0, T // 2, T - 300):
        ref = R.int8_gemm(xq[a:a + 300], sx[a:a + 300], wq, sw)
        R.within(out[a:a + 300], ref, REL * ref.abs() + R.TINY, f"rows {a}..")
    del out
    T, K, N = 40_000, 57_344, 64                        # T * K = 2.29e9 codes
    xq = torch.randint(-127, 128, (T, K), dtype=torch.int8, device=DEV)
    sx, wq, sw = R.scales(9, T).to(DEV), R.codes(10, N, K).to(DEV), R.scales(11, N, mean=1e-4).to(DEV)
    out = moe.moe_gemm_int8(xq, sx, wq, sw, _ws(1))
    for a in (0, T - 200):
        ref = R.int8_gemm(xq[a:a + 200], sx[a:a + 200], wq, sw)
        R.within(out[a:a + 200], ref, REL * ref.abs() + R.TINY, f"rows {a}..")


@pytest.mark.parametrize("T,K,N", [(1, 65536, 64), (5, 65536, 192), (300, 65536, 2304)])
def test_gemm_int8_extreme_sums(T, K, N):
    """Every code at its extreme, -128 included: sums of 2^30 stay exact."""
    xq = torch.full((T, K), -128, dtype=torch.int8)
    wq = torch.full((N, K), -128, dtype=torch.int8)
    wq[1::2] = 127
    sx, sw = torch.ones(T), torch.ones(N)
    sx[0] = 2.0 ** -40
    out = moe.moe_gemm_int8(xq.to(DEV), sx.to(DEV), wq.to(DEV), sw.to(DEV), _ws(T)).cpu()
    big, low = 2.0 ** 30, -128.0 * 127 * K
    want = torch.tensor([big if n % 2 == 0 else low for n in range(N)], dtype=R.D)[None, :] * sx.to(R.D)[:, None]
    R.within(out, want, R.BF16 * want.abs(), "extremes")
    assert (out[:, 0].double() == want[:, 0]).all()


def test_gemm_int8_special_scales():
    T, K, N = 5, 256, 128
    xq, sx, wq, sw = _dense(T, K, N, seed=77)
    sx[1], sx[2] = float("nan"), 0.0
    sw[3] = float("nan")
    out = moe.moe_gemm_int8(xq.to(DEV), sx.to(DEV), wq.to(DEV), sw.to(DEV), _ws(T)).cpu()
    assert torch.isnan(out[1]).all() and torch.isnan(out[:, 3]).all()
    keep = torch.ones(N, dtype=torch.bool)
    keep[3] = False
    assert (out[2, keep] == 0).all()
    ref = R.int8_gemm(xq, sx, wq, sw)
    R.within(out[4, keep], ref[4, keep], REL * ref[4, keep].abs(), "a plain row")


@pytest.mark.parametrize("T,K,N", [(5, 256, 128), (3, 7168, 2048), (700, 2048, 4096)])
def test_gemm_int8_scales_near_the_ends_of_the_range(T, K, N):
    """Rows quantised from values around 1e38 and 1e-30: the result is in range wherever its value is."""
    xq, sx, wq, sw = _dense(T, K, N, seed=78)
    sx[0], sx[1], sx[T - 1] = 2.6e36, 1e-32, 1e33
    sw *= 1e-4
    out = moe.moe_gemm_int8(xq.to(DEV), sx.to(DEV), wq.to(DEV), sw.to(DEV), _ws(T))
    ref = R.int8_gemm(xq.to(DEV), sx.to(DEV), wq.to(DEV), sw.to(DEV))
    assert ref.abs().max() < 3e38
    R.within(out, ref, REL * ref.abs() + R.TINY, "far scales")


def test_gemm_int8_empty_and_refusals():
    wq, sw = R.codes(1, 128, 256).to(DEV), R.scales(2, 128).to(DEV)
    ws = _ws(4)
    e = moe.moe_gemm_int8(torch.empty(0, 256, dtype=torch.int8, device=DEV), torch.empty(0, device=DEV), wq, sw, ws)
    assert e.shape == (0, 128)
    xq, sx = R.codes(3, 4, 256).to(DEV), R.scales(4, 4).to(DEV)
    with pytest.raises(AssertionError, match="Wq"):
        moe.moe_gemm_int8(xq, sx, wq[:, :192].contiguous(), sw, ws)
    with pytest.raises(AssertionError, match="sx"):
        moe.moe_gemm_int8(xq, sx[:3], wq, sw, ws)
    with pytest.raises(AssertionError, match="contiguous"):
        moe.moe_gemm_int8(xq, sx, wq.t().contiguous().t(), sw, ws)
    with pytest.raises(moe.MoEError):
        moe.moe_gemm_int8(xq[:, :96].contiguous(), sx, wq[:, :96].contiguous(), sw, ws)
    with pytest.raises(moe.MoEError, match="workspace"):
        moe.moe_gemm_int8(xq, sx, wq, sw, ws[:128])


# ---------------------------------------------------------------- one matrix an expert

def _grouped_check(counts, T, k, K, N, seed):
    E = len(counts)
    assert sum(counts) <= T * k
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    P, used = T * k, offsets[-1]
    xq, sx = R.codes(seed, P, K).to(DEV), R.scales(seed + 1, P).to(DEV)
    wq, sw = R.codes(seed + 2, E, N, K).to(DEV), R.scales(seed + 3, E, N, mean=0.001).to(DEV)
    t = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
    ws = _ws(T, E, k)
    out = torch.full((P + 2, N), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_grouped_gemm_int8(xq, sx, t(counts), t(offsets), wq, sw, T, k, ws, out=out[:P])
    assert moe.moe_get_device_error(ws) == 0
    for e, c in enumerate(counts):
        a, b = offsets[e], offsets[e + 1]
        if c:
            ref = R.int8_gemm(xq[a:b], sx[a:b], wq[e], sw[e])
            R.within(out[a:b], ref, REL * ref.abs() + R.TINY, f"expert {e} of {counts[:8]}")
    assert (out[used:] == 7.0).all(), "rows no expert has were written"


@pytest.mark.parametrize("counts,T,k,K,N", [
    ([1], 1, 1, 64, 64),
    ([0, 1, 0, 0], 1, 1, 2048, 192),
    ([0, 0, 0], 2, 2, 128, 128),                                  # every pair dropped
    ([3, 0, 17, 1, 0, 16, 32, 5], 40, 2, 448, 704),               # rows left over behind the last segment
    ([256, 257, 255, 1], 769, 1, 256, 320),
    ([1000, 0, 24], 512, 2, 1088, 2048),
    ([15, 33, 0, 64, 129, 300, 2, 1], 136, 4, 320, 4096),
    ([512, 511, 513, 500, 12, 0, 700, 1300], 506, 8, 2048, 1024),
])
def test_grouped_gemm_int8(counts, T, k, K, N):
    _grouped_check(counts, T, k, K, N, seed=len(counts) + K)


@pytest.mark.parametrize("pairs", [0, 1], indirect=True)
@pytest.mark.parametrize("counts,T,k,K,N", [
    ([0, 1, 0, 0], 1, 1, 2048, 192),
    ([3, 0, 17, 1, 0, 16, 32, 5], 40, 2, 448, 704),
    ([256, 257, 255, 1], 769, 1, 256, 320),
    ([512, 511, 513, 500, 12, 0, 700, 1300], 506, 8, 2048, 1024),
    ([0] * 511 + [7], 7, 1, 128, 64),
    ([2] * 512, 1024, 1, 128, 64),
])
def test_grouped_gemm_int8_every_form(pairs, counts, T, k, K, N):
    _grouped_check(counts, T, k, K, N, seed=K + N)


@pytest.mark.parametrize("T,E,k,alpha,K,N", [(32, 64, 8, 1.0, 2048, 1024), (3, 512, 8, 0.1, 256, 128),
                                             (700, 16, 4, 0.3, 1024, 768)])
def test_grouped_gemm_int8_routed(T, E, k, alpha, K, N):
    idx = wl.random_routing(T, E, k, alpha, seed=T)
    counts, _, _, _ = R.permutation(idx, E)
    _grouped_check(counts.tolist(), T, k, K, N, seed=E)


def test_grouped_gemm_int8_refuses_segments_outside_the_rows():
    """Counts and offsets are read on the device: segments past the rows set an error bit and write nothing."""
    T, k, K, N = 8, 2, 128, 128
    xq, sx = R.codes(1, 16, K).to(DEV), R.scales(2, 16).to(DEV)
    wq, sw = R.codes(3, 2, N, K).to(DEV), R.scales(4, 2, N).to(DEV)
    for counts, offsets in (([9, 9], [0, 9, 18]), ([4, 4], [0, 13, 17]), ([4, 4], [-4, 0, 4])):
        ws = _ws(T, 2, k)
        out = torch.full((T * k, N), 7.0, dtype=torch.bfloat16, device=DEV)
        t = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
        moe.moe_grouped_gemm_int8(xq, sx, t(counts), t(offsets), wq, sw, T, k, ws, out=out)
        assert moe.moe_get_device_error(ws) == moe.DEVERR_PLAN
        assert (out == 7.0).all()
        # the workspace is usable afterwards
        moe.moe_clear_device_error(ws)
        moe.moe_grouped_gemm_int8(xq, sx, t([10, 6]), t([0, 10, 16]), wq, sw, T, k, ws, out=out)
        assert moe.moe_get_device_error(ws) == 0
        ref = R.int8_gemm(xq[10:], sx[10:], wq[1], sw[1])
        R.within(out[10:], ref, REL * ref.abs() + R.TINY, "after a refusal")
