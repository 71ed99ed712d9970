"""The norm, int8 product and sorted-row operators together, as they are used: an int8 expert block in serving
(eager, on another stream, captured into a graph and replayed), and a training step's forward and backward pass
(marked gpu)."""

from __future__ import annotations

import pytest
import torch

from grouped_gemm_02_b200 import moe
from grouped_gemm_02_b200 import workload as wl
from tests import ops_helpers as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-5


class Int8Block:
    """norm -> int8 codes -> sort -> expert product -> weighted return, on buffers that a program keeps."""

    def __init__(self, T, d, N, E, k, seed):
        self.T, self.k, self.E = T, k, E
        self.w = (1 + 0.2 * torch.randn(d, generator=R.gen(seed))).to(torch.bfloat16).to(DEV)
        self.Wq, self.sw = moe.moe_quantize_int8_rows(R.randn(seed + 1, E, N, d, std=d ** -0.5).to(DEV))
        self.ws = moe.new_workspace(T, 64, 64, E, k)

    def __call__(self, x, r, idx, gates, stream=None):
        q, s, xsum = moe.moe_rmsnorm_int8(x, self.w, EPS, residual=r, stream=stream)
        c, o, perm, inv, xpq, sxp = moe.moe_permute_int8(idx, q, s, self.E, self.ws, stream=stream)
        y = moe.moe_grouped_gemm_int8(xpq, sxp, c, o, self.Wq, self.sw, self.T, self.k, self.ws, stream=stream)
        return moe.moe_combine_weighted(y, inv, gates, stream=stream), xsum

    def reference(self, x, r, idx, gates):
        """The same steps in 64 bits from the same int8 codes: what is left is the product's and the return's rounding."""
        q, s, _ = moe.moe_rmsnorm_int8(x, self.w, EPS, residual=r)
        T, k = idx.shape
        out = torch.zeros(T, self.Wq.shape[1], dtype=R.D, device=DEV)
        mag = torch.zeros_like(out)
        for t in range(T):
            for j in range(k):
                e = int(idx[t, j])
                row = R.int8_gemm(q[t:t + 1], s[t:t + 1], self.Wq[e], self.sw[e])[0] * gates[t, j].double()
                out[t] += row
                mag[t] += row.abs()
        return out, mag


def _inputs(T, d, E, k, seed):
    x, r = R.randn(seed, T, d).to(DEV), R.randn(seed + 1, T, d).to(DEV)
    return x, r, wl.random_routing(T, E, k, 0.5, seed).to(DEV), wl.random_gates(T, k, seed).to(DEV)


@pytest.mark.parametrize("T,d,N,E,k", [(1, 256, 192, 8, 2), (37, 512, 320, 16, 4), (300, 1024, 256, 4, 4)])
def test_int8_block(T, d, N, E, k):
    blk = Int8Block(T, d, N, E, k, seed=3)
    args = _inputs(T, d, E, k, seed=5)
    out, xsum = blk(*args)
    assert torch.equal(xsum, R.add_bf16(args[0], args[1]))
    ref, mag = blk.reference(*args)
    # an expert row is rounded to bf16 before the return: half a step of every term, then one of the sum
    R.within(out, ref, R.BF16 * (1 + R.BF16) * mag + R.BF16 * ref.abs() + 24 * R.F32 * mag, "int8 block")
    assert moe.moe_get_device_error(blk.ws) == 0


def test_int8_block_on_another_stream():
    T, d, N, E, k = 64, 512, 320, 16, 4
    blk = Int8Block(T, d, N, E, k, seed=7)
    args = _inputs(T, d, E, k, seed=8)
    want, wsum = blk(*args)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        out, xsum = blk(*args, stream=st)
    st.synchronize()
    assert torch.equal(out, want) and torch.equal(xsum, wsum)
    with torch.cuda.stream(st):
        out, xsum = blk(*args)
    st.synchronize()
    assert torch.equal(out, want) and torch.equal(xsum, wsum)


def test_int8_blocks_side_by_side():
    """Two blocks with a workspace each, in flight on two streams at once."""
    shapes = [(96, 512, 320, 16, 4), (257, 256, 448, 8, 2)]
    blks = [Int8Block(*s, seed=9 + i) for i, s in enumerate(shapes)]
    args = [_inputs(s[0], s[1], s[3], s[4], seed=20 + i) for i, s in enumerate(shapes)]
    want = [b(*a)[0] for b, a in zip(blks, args)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in shapes]
    got = [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            got[i].append(blks[i](*args[i], stream=st)[0])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


def test_int8_block_captured_and_replayed():
    T, d, N, E, k = 48, 512, 320, 16, 4
    blk = Int8Block(T, d, N, E, k, seed=11)
    a, b = _inputs(T, d, E, k, seed=12), _inputs(T, d, E, k, seed=13)
    want = [blk(*v)[0].clone() for v in (a, b)]
    static = [t.clone() for t in a]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, xsum = blk(*static)
    for v, w in ((a, want[0]), (b, want[1]), (a, want[0])):
        for s, t in zip(static, v):
            s.copy_(t)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)


def _train(x, r, w, W, idx, gates, inv, perm, dout, ds):
    """norm -> sort -> expert product (bf16 values, fp32 matmul) -> weighted return, and back by the framework's
    gradients; the expert product's own gradient is torch's."""
    T, k = gates.shape
    y, xsum = moe.moe_rmsnorm(x, w, EPS, residual=r)
    tok = perm.long() // k
    e = idx.reshape(-1)[perm.long()].long()
    xp = y[tok]
    yp = torch.bmm(xp.float()[:, None, :], W[e])[:, 0].to(torch.bfloat16)
    out = moe.moe_combine_weighted(yp, inv, gates)
    dyp, dgate = moe.moe_combine_weighted_backward(dout, yp, inv, gates)
    dxp = torch.bmm(dyp.float()[:, None, :], W[e].transpose(1, 2))[:, 0].to(torch.bfloat16)
    dy = moe.moe_permute_backward(dxp, inv, T, k)
    dx, dw = moe.moe_rmsnorm_backward(dy, xsum, w, EPS, dxsum=ds)
    return out, dgate, dx, dw


def _train_case(T=37, d=128, E=8, k=3):
    x, r, idx, gates = _inputs(T, d, E, k, seed=31)
    w = (1 + 0.2 * torch.randn(d, generator=R.gen(33))).to(torch.bfloat16).to(DEV)
    W = (torch.randn(E, d, d, generator=R.gen(34)) * d ** -0.5).to(DEV)
    _, _, perm, inv = (t.to(DEV) for t in R.permutation(idx, E))
    dout, ds = R.randn(35, T, d).to(DEV), R.randn(36, T, d, std=0.5).to(DEV)
    return x, r, w, W, idx, gates, inv, perm, dout, ds


def test_training_step_gradients():
    """Against automatic differentiation of the whole block in 64 bits.  Relative 2-norm error: five bf16 roundings
    lie between an input and a gradient (y, yp, dyp, dxp, dy or dx), each at most 2^-8 of its value: below 5 * 2^-8."""
    x, r, w, W, idx, gates, inv, perm, dout, ds = case = _train_case()
    out, dgate, dx, dw = _train(*case)
    leaf = lambda t: t.to(R.D).detach().requires_grad_(True)
    s, w64, g64 = leaf(R.add_bf16(x, r)), leaf(w), leaf(gates)
    y = R.rmsnorm(s, w64, EPS)
    ref = sum(g64[:, j:j + 1] * torch.bmm(y[:, None, :], W.to(R.D)[idx[:, j].long()])[:, 0] for j in range(idx.shape[1]))
    gs, gw, gg = torch.autograd.grad((ref * dout.to(R.D)).sum() + (s * ds.to(R.D)).sum(), (s, w64, g64))
    for got, want, what in ((out, ref, "out"), (dgate, gg, "dgate"), (dx, gs, "dx"), (dw, gw, "dw")):
        rel = (got.to(R.D) - want).norm() / want.norm()
        assert float(rel.detach()) < 5 * R.BF16, (what, float(rel.detach()))


def test_training_step_captured_beside_an_eager_one():
    """A captured step replays what an eager one of the same buffers computes, while that one's results live."""
    case = _train_case()
    eager = _train(*case)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = _train(*case)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager, captured):
        assert torch.equal(a, b)
