"""Rows sorted by expert and back with the gates applied, and the gradient of both, on the GPU (marked gpu).

Sorting copies: exact.  A return adds at most 9 fp32 terms (each product and each addition a rounding:
18 * 2^-24 of the sum of magnitudes) and rounds once (2^-8).  A dot product adds at most
ceil(d / (8 * 32)) * 8 products in a thread and 5 + 8 more levels: 2^-24 a step of the sum of magnitudes."""

from __future__ import annotations

import pytest
import torch

from grouped_gemm_02_b200 import moe
from grouped_gemm_02_b200 import workload as wl
from tests import ops_helpers as R

pytestmark = pytest.mark.gpu
DEV = "cuda"

SIZES = [(1, 4, 1, 64), (1, 256, 8, 7168), (2, 2, 2, 192), (7, 8, 3, 1088), (32, 64, 8, 2048), (128, 8, 8, 64),
         (129, 8, 8, 320), (333, 384, 8, 448), (700, 16, 5, 4096), (2049, 512, 2, 128), (3, 3, 1, 16384),
         (301, 8, 1, 7168), (299, 8, 2, 4096), (303, 4, 4, 2112), (777, 8, 1, 64), (402, 8, 3, 256), (1023, 8, 8, 256)]


def _routing(T, E, k, seed, bad=()):
    idx = wl.random_routing(T, E, k, 0.5, seed=seed)
    for t, j, v in bad:
        idx[t, j] = v
    return idx


def _case(T, E, k, seed, drop=False):
    bad = [(0, 0, E), (T // 2, k - 1, -1), (T - 1, 0, 1 << 20)] if drop else ()
    idx = _routing(T, E, k, seed, bad)
    _, _, _, inv = R.permutation(idx, E)
    w = wl.random_gates(T, k, seed)
    return idx, inv, w


@pytest.mark.parametrize("drop", [False, True])
@pytest.mark.parametrize("T,E,k,d", SIZES)
def test_permute_int8(T, E, k, d, drop):
    idx, inv, _ = _case(T, E, k, seed=T, drop=drop)
    counts, offsets, perm, inv = R.permutation(idx, E)
    xq, sx = R.codes(1, T, d), R.scales(2, T)
    ws = moe.new_workspace(T, 64, 64, E, k)
    got = moe.moe_permute_int8(idx.to(DEV), xq.to(DEV), sx.to(DEV), E, ws)
    n = int(offsets[E])
    assert moe.moe_get_device_error(ws) == (moe.DEVERR_EXPERT_RANGE if drop else 0)
    g = [t.cpu() for t in got]
    assert torch.equal(g[0], counts) and torch.equal(g[1], offsets) and torch.equal(g[3], inv)
    assert torch.equal(g[2][:n], perm)
    tok = perm.long() // k
    assert torch.equal(g[4][:n], xq[tok]) and torch.equal(g[5][:n], sx[tok])


@pytest.mark.parametrize("T", [3, 128, 500])
def test_permute_int8_of_one_expert_chosen_more_than_once(T):
    """The same expert in several of a token's places: every pair keeps a position of its own, in order."""
    E, k, d = 8, 4, 128
    idx = torch.full((T, k), 5, dtype=torch.int32)
    idx[:, 1] = 2
    counts, offsets, perm, inv = R.permutation(idx, E)
    xq, sx = R.codes(25, T, d), R.scales(26, T)
    ws = moe.new_workspace(T, 64, 64, E, k)
    g = [t.cpu() for t in moe.moe_permute_int8(idx.to(DEV), xq.to(DEV), sx.to(DEV), E, ws)]
    assert torch.equal(g[0], counts) and torch.equal(g[1], offsets) and torch.equal(g[2], perm) and torch.equal(g[3], inv)
    assert torch.equal(g[4], xq[perm.long() // k]) and torch.equal(g[5], sx[perm.long() // k])
    wq, sw = R.codes(27, E, 128, d).to(DEV), R.scales(28, E, 128, mean=0.001).to(DEV)
    out = moe.moe_grouped_gemm_int8(*(t.to(DEV) for t in (g[4], g[5], g[0], g[1])), wq, sw, T, k, ws)
    ref = R.int8_gemm(g[4][T:].to(DEV), g[5][T:].to(DEV), wq[5], sw[5])
    R.within(out[T:], ref, (R.BF16 + 2.0 ** -21) * ref.abs() + R.TINY, "the chosen expert")


@pytest.mark.parametrize("T", [32768, 32769, 45000])
def test_permute_int8_of_many_pairs(T):
    """Around 2^18 pairs, where another way of finding the positions takes over."""
    E, k, d = 24, 8, 64
    idx = torch.randint(0, E, (T, k), generator=R.gen(T), dtype=torch.int32)
    idx[5, 3], idx[T - 1, 7] = E, -2
    xq, sx = R.codes(20, T, d), R.scales(21, T)
    ws = moe.new_workspace(T, 64, 64, E, k)
    got = [t.cpu() for t in moe.moe_permute_int8(idx.to(DEV), xq.to(DEV), sx.to(DEV), E, ws)]
    assert moe.moe_get_device_error(ws) == moe.DEVERR_EXPERT_RANGE
    flat = idx.reshape(-1).long()
    ok = (flat >= 0) & (flat < E)
    key, perm = torch.sort(torch.where(ok, flat, torch.full_like(flat, E)), stable=True)
    n = int(ok.sum())
    perm = perm[:n]
    counts = torch.bincount(key[:n], minlength=E)
    assert torch.equal(got[0].long(), counts) and torch.equal(got[1].long(), torch.cat([counts.new_zeros(1), counts.cumsum(0)]))
    inv = torch.full((T * k,), -1, dtype=torch.int64)
    inv[perm] = torch.arange(n)
    assert torch.equal(got[2][:n].long(), perm) and torch.equal(got[3].long(), inv)
    assert torch.equal(got[4][:n], xq[perm // k]) and torch.equal(got[5][:n], sx[perm // k])


def test_sorted_rows_past_32_bit_offsets():
    """Rows whose offsets pass 2^31 elements: the last positions, where an overflow would show."""
    T, E, k, d = 40_000, 8, 8, 7168                          # T * k * d = 2.29e9
    idx = torch.stack([torch.arange(E, dtype=torch.int32)] * T)
    xq = torch.randint(-127, 128, (T, d), dtype=torch.int8, device=DEV)
    sx = R.scales(22, T).to(DEV)
    ws = moe.new_workspace(T, 64, 64, E, k)
    counts, offsets, perm, inv, xpq, sxp = moe.moe_permute_int8(idx.to(DEV), xq, sx, E, ws)
    for pos in (0, T * k // 2 + 17, T * k - 1):
        t = int(perm[pos]) // k
        assert torch.equal(xpq[pos], xq[t]) and float(sxp[pos]) == float(sx[t])
    del xpq
    y = torch.empty(T * k, d, dtype=torch.bfloat16, device=DEV)
    y.copy_(torch.arange(T * k, device=DEV)[:, None].remainder(251))
    w = wl.random_gates(T, k, 23).to(DEV)
    dout = R.randn(24, T, d).to(DEV)
    out = moe.moe_combine_weighted(y, inv, w)
    dx = moe.moe_permute_backward(y, inv, T, k)
    for t in (0, T // 2 + 3, T - 1):
        rows = inv.view(T, k)[t].long()
        ref = (y[rows].double() * w[t].double()[:, None]).sum(0)
        R.within(out[t], ref, R.BF16 * ref + 18 * R.F32 * ref, "combine")
        ref = y[rows].double().sum(0)
        R.within(dx[t], ref, R.BF16 * ref + 18 * R.F32 * ref, "permute backward")
    dy, dw = moe.moe_combine_weighted_backward(dout, y, inv, w, dy_p=y)
    for t in (0, T - 1):
        rows = inv.view(T, k)[t].long()
        ref = w[t].double()[:, None] * dout[t].double()
        R.within(dy[rows], ref, (R.BF16 + R.F32) * ref.abs() + R.TINY, "dy_p")


def test_permute_int8_agrees_with_moe_permute():
    T, E, k, d = 515, 64, 8, 256
    idx = _routing(T, E, k, 9).to(DEV)
    x = R.randn(3, T, d).to(DEV)
    ws = moe.new_workspace(T, d, 64, E, k)
    a = moe.moe_permute(idx, x, E, ws)
    xq, sx = moe.moe_quantize_int8_rows(x)
    b = moe.moe_permute_int8(idx, xq, sx, E, ws)
    for u, v in zip(a[:4], b[:4]):
        assert torch.equal(u, v)
    q, s = moe.moe_quantize_int8_rows(a[4])
    assert torch.equal(q, b[4]) and torch.equal(s, b[5])


@pytest.mark.parametrize("drop", [False, True])
@pytest.mark.parametrize("with_shared", [False, True])
@pytest.mark.parametrize("T,E,k,d", SIZES)
def test_combine_weighted(T, E, k, d, with_shared, drop):
    idx, inv, w = _case(T, E, k, seed=T + 1, drop=drop)
    y = R.randn(4, T * k, d)
    sh = R.randn(5, T, d) if with_shared else None
    out = moe.moe_combine_weighted(y.to(DEV), inv.to(DEV), w.to(DEV), shared_out=None if sh is None else sh.to(DEV))
    ref, mag = R.combine(y, inv, w, sh)
    R.within(out, ref, R.BF16 * ref.abs() + 18 * R.F32 * mag + R.TINY, "combine")


@pytest.mark.parametrize("drop", [False, True])
@pytest.mark.parametrize("T,E,k,d", SIZES)
def test_combine_weighted_backward(T, E, k, d, drop):
    idx, inv, w = _case(T, E, k, seed=T + 2, drop=drop)
    y, dout = R.randn(6, T * k, d), R.randn(7, T, d, std=0.1)
    dy = torch.full((T * k, d), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_combine_weighted_backward(dout.to(DEV), y.to(DEV), inv.to(DEV), w.to(DEV), dy_p=dy)
    dy2, dw = moe.moe_combine_weighted_backward(dout.to(DEV), y.to(DEV), inv.to(DEV), w.to(DEV))
    rdy, rdw, mag = R.combine_grad(dout, y, inv, w)
    pos = inv.long()
    has = pos >= 0
    want = rdy[has]
    for got in (dy, dy2):
        R.within(got.cpu()[pos[has]], want, (R.BF16 + R.F32) * want.abs() + R.TINY, "dy_p")
    steps = -(-d // 256) * 8 + 13
    R.within(dw, rdw, steps * R.F32 * mag + R.TINY, "dw")
    assert (dw.cpu().reshape(-1)[~has] == 0).all()
    free = torch.ones(T * k, dtype=torch.bool)
    free[pos[has]] = False
    assert (dy.cpu()[free] == 7.0).all(), "rows no pair has were written"


def test_combine_weighted_backward_in_place():
    T, E, k, d = 65, 8, 3, 320
    _, inv, w = _case(T, E, k, seed=8)
    y, dout = R.randn(9, T * k, d).to(DEV), R.randn(10, T, d).to(DEV)
    dy, dw = moe.moe_combine_weighted_backward(dout, y, inv.to(DEV), w.to(DEV))
    y1 = y.clone()
    dy1, dw1 = moe.moe_combine_weighted_backward(dout, y1, inv.to(DEV), w.to(DEV), dy_p=y1)
    assert dy1 is y1 and torch.equal(dy, dy1) and torch.equal(dw, dw1)


@pytest.mark.parametrize("drop", [False, True])
@pytest.mark.parametrize("with_addend", [False, True])
@pytest.mark.parametrize("T,E,k,d", SIZES)
def test_permute_backward(T, E, k, d, with_addend, drop):
    idx, inv, w = _case(T, E, k, seed=T + 3, drop=drop)
    dxp = R.randn(11, T * k, d)
    add = R.randn(12, T, d) if with_addend else None
    dx = moe.moe_permute_backward(dxp.to(DEV), inv.to(DEV), T, k, addend=None if add is None else add.to(DEV))
    ref, mag = R.combine(dxp, inv, torch.ones(T, k), add)
    R.within(dx, ref, R.BF16 * ref.abs() + 18 * R.F32 * mag + R.TINY, "dx")
    if with_addend:
        buf = add.to(DEV)
        moe.moe_permute_backward(dxp.to(DEV), inv.to(DEV), T, k, addend=buf, dx=buf)
        assert torch.equal(buf, dx)
    else:
        assert torch.equal(dx, moe.moe_combine(dxp.to(DEV), inv.to(DEV), T, k))


def test_positions_outside_the_rows_are_dropped():
    """inv_perm comes from the caller: a position past the rows adds nothing and writes nothing."""
    T, k, d = 4, 2, 128
    inv = torch.tensor([0, 1, 8, 3, 1 << 30, 5, -5, 7], dtype=torch.int32)
    ok = torch.where((inv >= 0) & (inv < 8), inv, torch.full_like(inv, -1))
    y, w, dout = R.randn(13, 8, d), wl.random_gates(T, k, 14), R.randn(15, T, d)
    out = moe.moe_combine_weighted(y.to(DEV), inv.to(DEV), w.to(DEV))
    ref, mag = R.combine(y, ok, w)
    R.within(out, ref, R.BF16 * ref.abs() + 18 * R.F32 * mag + R.TINY, "combine")
    dy = torch.full((9, d), 7.0, dtype=torch.bfloat16, device=DEV)
    _, dw = moe.moe_combine_weighted_backward(dout.to(DEV), y.to(DEV), inv.to(DEV), w.to(DEV), dy_p=dy[:8])
    assert (dw.cpu().reshape(-1)[ok < 0] == 0).all()
    assert (dy.cpu()[[2, 4, 6, 8]] == 7.0).all()


def test_non_finite_rows_of_dropped_pairs_add_nothing():
    T, k, d = 2, 2, 64
    inv = torch.tensor([0, -1, 1, 2], dtype=torch.int32)
    y = R.randn(16, 4, d)
    y[3] = float("nan")
    w = torch.tensor([[0.5, float("nan")], [0.25, 0.75]])
    out = moe.moe_combine_weighted(y.to(DEV), inv.to(DEV), w.to(DEV)).cpu()
    assert torch.equal(out[0], (y[0].float() * 0.5).to(torch.bfloat16)) and torch.isfinite(out).all()


def test_empty_batch_and_refusals():
    b = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=DEV)
    i = lambda n: torch.empty(n, dtype=torch.int32, device=DEV)
    w = torch.empty(0, 2, device=DEV)
    assert moe.moe_combine_weighted(b(0, 64), i(0), w).shape == (0, 64)
    dy, dw = moe.moe_combine_weighted_backward(b(0, 64), b(0, 64), i(0), w)
    assert dy.shape == (0, 64) and dw.shape == (0, 2)
    assert moe.moe_permute_backward(b(0, 64), i(0), 0, 2).shape == (0, 64)
    ws = moe.new_workspace(4, 64, 64, 8, 2)
    got = moe.moe_permute_int8(torch.empty(0, 2, dtype=torch.int32, device=DEV),
                               torch.empty(0, 64, dtype=torch.int8, device=DEV), torch.empty(0, device=DEV), 8, ws)
    assert (got[0] == 0).all() and (got[1] == 0).all() and got[4].shape == (0, 64)
    with pytest.raises(AssertionError, match="inv_perm"):
        moe.moe_combine_weighted(b(4, 64), i(3), torch.empty(2, 2, device=DEV))
    with pytest.raises(AssertionError, match="y_p"):
        moe.moe_combine_weighted(b(3, 64), i(4), torch.empty(2, 2, device=DEV))
    with pytest.raises(AssertionError, match="topk_w"):
        moe.moe_combine_weighted(b(4, 64), i(4), torch.empty(2, 2, device=DEV, dtype=torch.bfloat16))
    with pytest.raises(moe.MoEError):
        moe.moe_combine_weighted(b(4, 96), i(4), torch.empty(2, 2, device=DEV))
