"""Plain 64-bit definitions of the norm, the int8 product and the sorted-row operators, for their tests.

Tolerances count roundings: half a step of the type, eps / 2 relative (bf16 2^-8, fp32 2^-24), plus the
fp32 steps before it, each at most 2^-24 of the magnitudes it adds."""

from __future__ import annotations

import torch

BF16, F32 = 2.0 ** -8, 2.0 ** -24
TINY = 2.0 ** -126          # results in the subnormal range are held to absolute steps
D = torch.float64


def within(got: torch.Tensor, ref: torch.Tensor, tol: torch.Tensor, what: str):
    got, ref, tol = got.to(D).cpu(), ref.to(D).cpu(), tol.to(D).cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    both_nan = torch.isnan(got) & torch.isnan(ref)
    bad = ~((got - ref).abs() <= tol) & ~both_nan & ~((got == ref) & torch.isinf(ref))
    if bad.any():
        i = tuple(int(v[0]) for v in bad.nonzero(as_tuple=True))
        raise AssertionError(f"{what}: {int(bad.sum())} of {got.numel()} out of tolerance, first at {i}: "
                             f"{float(got[i]):.9g} against {float(ref[i]):.9g} (tolerance {float(tol[i]):.3g})")


def add_bf16(x, r):
    """bf16(x + r): the fp32 sum rounded to bf16, as the operator defines the stream."""
    return (x.float() + r.float()).to(torch.bfloat16)


def rmsnorm(s, w, eps):
    s = s.to(D)
    return s / torch.sqrt(s.square().mean(1, keepdim=True) + eps) * w.to(D)


def rmsnorm_grad(dy, s, w, eps, ds=None):
    """dx, dw and the magnitudes their sums run over."""
    dy, s, w = dy.to(D), s.to(D), w.to(D)
    rstd = 1 / torch.sqrt(s.square().mean(1, keepdim=True) + eps)
    n, g = s * rstd, dy * w
    dx = (g - n * (g * n).mean(1, keepdim=True)) * rstd
    mag = (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True)) * rstd
    if ds is not None:
        dx, mag = dx + ds.to(D), mag + ds.to(D).abs()
    return dx, (dy * n).sum(0), mag, (dy * n).abs().sum(0)


def int8_rows(y):
    """codes before rounding and scales of rows (finite, not below 2^-100)."""
    y = y.to(D)
    amax = y.abs().amax(1, keepdim=True)
    scale = torch.where(amax > 0, amax / 127, torch.ones_like(amax))
    return y / scale, scale[:, 0]


def int8_gemm(xq, sx, wq, sw):
    return (xq.to(D) @ wq.to(D).t()) * sx.to(D)[:, None] * sw.to(D)


def permutation(idx, E):
    """counts, offsets, perm, inv_perm with ids outside [0, E) dropped (numpy-free, on the CPU)."""
    flat = idx.reshape(-1).cpu().tolist()
    order = sorted((q for q, e in enumerate(flat) if 0 <= e < E), key=lambda q: (flat[q], q))
    inv = [-1] * len(flat)
    counts = [0] * E
    for pos, q in enumerate(order):
        inv[q] = pos
        counts[flat[q]] += 1
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    t = lambda v: torch.tensor(v, dtype=torch.int32)
    return t(counts), t(offsets), t(order), t(inv)


def combine(y, inv, w, shared=None):
    """out and the sum of magnitudes; inv [T*k] with -1 for dropped pairs."""
    T, k = w.shape
    pos = inv.view(T, k).long()
    has = (pos >= 0).to(D)[:, :, None]
    rows = torch.where(has > 0, y.to(D)[pos.clamp(min=0)], torch.zeros((), dtype=D, device=y.device))
    term = w.to(D)[:, :, None] * rows
    term = torch.where(has > 0, term, torch.zeros_like(term))
    out, mag = term.sum(1), term.abs().sum(1)
    if shared is not None:
        out, mag = out + shared.to(D), mag + shared.to(D).abs()
    return out, mag


def combine_grad(dout, y, inv, w):
    """dy rows by pair [T*k, d], dw [T, k] and dw's magnitudes."""
    T, k = w.shape
    pos = inv.view(T, k).long()
    has = pos >= 0
    rows = torch.where(has[:, :, None], y.to(D)[pos.clamp(min=0)], torch.zeros((), dtype=D, device=y.device))
    prod = dout.to(D)[:, None, :] * rows
    prod = torch.where(has[:, :, None], prod, torch.zeros_like(prod))
    dy = w.to(D)[:, :, None] * dout.to(D)[:, None, :]
    return dy.reshape(T * k, -1), prod.sum(2), prod.abs().sum(2)


def gen(seed, device="cpu"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def randn(seed, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen(seed)) * std).to(torch.bfloat16)


def codes(seed, *shape, lo=-127, hi=127):
    return torch.randint(lo, hi + 1, shape, generator=gen(seed), dtype=torch.int32).to(torch.int8)


def scales(seed, *shape, mean=0.03):
    return (torch.rand(*shape, generator=gen(seed)) + 0.5) * mean
