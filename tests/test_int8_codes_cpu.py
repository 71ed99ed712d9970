"""The int8 codes of a row against v * 127 / max|v| rounded to nearest, ties to even, for every bf16 mantissa of
the largest magnitude and of the value (CPU).

127 v is exact in 64 bits and so is the only tie, 63.5 at half the largest magnitude: any other quotient lies
at least 2^-17 from one (its denominator is below 2^8 times the power of two between the two exponents, which is
at most 2^8 where the quotient reaches 0.5), so rounding the 64-bit quotient gives the definition's code."""

import ctypes as C
import os
import subprocess

import numpy as np
import pytest


@pytest.fixture(scope="module")
def codes_of(tmp_path_factory):
    here = os.path.dirname(os.path.abspath(__file__))
    out = str(tmp_path_factory.mktemp("code") / "libcode.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-ffp-contract=off", "-o", out,
                    os.path.join(here, "int8_code_harness.cpp"), "-lm"], check=True)
    lib = C.CDLL(out)
    fp, ip = C.POINTER(C.c_float), C.POINTER(C.c_int)
    lib.int8_codes_of.argtypes = [C.c_float, fp, C.c_int, fp, fp, ip]

    def f(amax, v):
        v = np.ascontiguousarray(v, dtype=np.float32)
        scale, inv, q = C.c_float(), C.c_float(), np.empty(v.size, dtype=np.int32)
        lib.int8_codes_of(float(amax), v.ctypes.data_as(fp), v.size, C.byref(scale), C.byref(inv), q.ctypes.data_as(ip))
        return scale.value, inv.value, q
    return f


@pytest.mark.parametrize("exponent", [-107, -60, 0, 13, 120])
def test_codes_of_every_mantissa(codes_of, exponent):
    m = np.arange(128, 256, dtype=np.float64)
    v = np.concatenate([m * 2.0 ** -s for s in range(11)])
    v = np.concatenate([v, -v, [0.0]])
    for top in m:
        row = v[np.abs(v) <= top] * 2.0 ** exponent
        amax = top * 2.0 ** exponent
        scale, inv, q = codes_of(amax, row)
        want = np.round(127.0 * (row / 2.0 ** exponent) / top)
        assert np.array_equal(q, want), (top, row[q != want][:4], q[q != want][:4], want[q != want][:4])
        assert np.abs(q).max() == 127
        assert abs(scale / (amax / 127.0) - 1) <= 2.0 ** -24


def test_rows_without_a_scale(codes_of):
    for bits in (0x7F800000, 0x7FC00000):
        amax = np.array([bits], dtype=np.uint32).view(np.float32)[0]
        scale, inv, _ = codes_of(amax, [1.0])
        assert np.isnan(scale) and inv == 0.0
    for amax in (0.0, 2.0 ** -101, 255 * 2.0 ** -108):
        assert codes_of(amax, [amax])[:2] == (1.0, 0.0)
