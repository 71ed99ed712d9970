"""What the host computes on several threads is what it computes on one (CPU): the oracle's row ranges and the
weights' draws."""

import ctypes as C

import numpy as np
import pytest
import torch

import oracle
from grouped_gemm_02_b200 import workload as wl


def _bits(*shape, seed=0):
    return wl.bf16_bits(wl._normal_bf16(shape, 1.0, seed, "bits", "cpu"))


def _p(a, ct):
    return a.ctypes.data_as(C.POINTER(ct))


@pytest.fixture(params=[1, 3, 16])
def threads(request, monkeypatch):
    monkeypatch.setattr(oracle, "default_threads", lambda: request.param)


@pytest.mark.parametrize("R", [1, 513, 1000])
def test_row_quantisers_in_parts(threads, R):
    x, L = _bits(R, 2048, seed=R), oracle.lib()
    for fn, block, f in ((L.oracle_quantize_rows_fp8, 128, oracle.quantize_rows_fp8),
                         (L.oracle_quantize_rows_fp4, 32, oracle.quantize_rows_fp4)):
        q, s = np.empty((R, 2048), np.uint8), np.empty((R, 2048 // block))
        assert fn(_p(x, C.c_uint16), R, 2048, _p(q, C.c_uint8), _p(s, C.c_double)) == 0
        got = f(x)
        assert np.array_equal(got[0], q) and np.array_equal(got[1], s)


def test_block_quantiser_router_and_h_in_parts(threads):
    L, d, f, T, E = oracle.lib(), 1024, 1152, 40, 24
    W = _bits(f, d, seed=1)
    q, s = np.empty((f, d), np.uint8), np.empty((f // 128, d // 128))
    assert L.oracle_quantize_blocks_fp8(_p(W, C.c_uint16), f, d, _p(q, C.c_uint8), _p(s, C.c_double)) == 0
    got = oracle.quantize_blocks_fp8(W)
    assert np.array_equal(got[0], q) and np.array_equal(got[1], s)
    x, Wg, bias = _bits(T, d, seed=2), _bits(E, d, seed=3), np.arange(E, dtype=np.float32)
    ref = np.empty((T, E))
    assert L.oracle_router_logits(_p(x, C.c_uint16), _p(Wg, C.c_uint16), _p(bias, C.c_float), T, d, E, _p(ref, C.c_double)) == 0
    assert np.array_equal(oracle.router_logits(x, Wg, bias), ref)
    xq, sx = oracle.quantize_rows_fp8(x[:1])
    hq, sh = np.empty(f, np.uint8), np.empty(f // 128)
    assert L.oracle_expert_h_fp8(_p(q, C.c_uint8), _p(s, C.c_double), _p(q, C.c_uint8), _p(s, C.c_double),
                                 _p(xq, C.c_uint8), _p(sx, C.c_double), d, f, _p(hq, C.c_uint8), _p(sh, C.c_double)) == 0
    got = oracle.expert_h_fp8(xq, sx, q, s, q, s)
    assert np.array_equal(got[0], hq) and np.array_equal(got[1], sh)


def test_a_part_that_fails_is_reported(threads):
    with pytest.raises(oracle.OracleError):
        oracle.quantize_blocks_fp8(_bits(4 * 128 + 64, 2048))


def test_weights_drawn_together():
    s = wl.TINY.with_(E=5)
    w = wl.make_weights(s, seed=4)
    for n, shape, k in (("W1", (s.E, s.f, s.d), s.d), ("W3", (s.E, s.f, s.d), s.d), ("W2", (s.E, s.d, s.f), s.f)):
        assert torch.equal(w[n], wl._normal_bf16(shape, k ** -0.5, 4, n, "cpu"))
