"""Codes and scales of 8 bits from the reciprocal and one exact remainder (rows_out.h):
the same as from divisions, checked over all significands (CPU; a C compiler)."""
import ctypes
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
needs_gcc = pytest.mark.skipif(shutil.which("gcc") is None, reason="no C compiler")


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("quotients") / "quotients.so")
    subprocess.check_call(["gcc", "-O3", "-march=native", "-fno-fast-math", "-ffp-contract=off", "-fno-math-errno", "-fopenmp", "-shared", "-fPIC",
                           "-Wall", "-o", out, os.path.join(HERE, "quotients.c"), "-lm"])
    so = ctypes.CDLL(out)
    so.other_sides.restype = so.other_scales.restype = ctypes.c_longlong
    so.other_sides.argtypes = [ctypes.c_long, ctypes.c_long, ctypes.c_int, ctypes.c_int]
    so.other_scales.argtypes = [ctypes.c_float, ctypes.c_int]
    return so


@needs_gcc
def test_codes_of_the_divided_quotient(lib):
    # Midpoints of 5 bits between E4M3 values and of 8 bits, k + 1/2 up to 128, for
    # Q8_0; the former are among the latter.
    assert lib.other_sides(1 << 23, 1 << 24, 8, 1) == 0


@needs_gcc
def test_scales_are_the_divided_ones(lib):
    assert lib.other_scales(448.0, 1) == 0 and lib.other_scales(127.0, 1) == 0


@needs_gcc
def test_the_check_sees_a_missing_remainder(lib):
    assert lib.other_sides(1 << 23, (1 << 23) + 1000, 5, 0) > 0
    assert lib.other_scales(448.0, 0) > 0 and lib.other_scales(127.0, 0) > 0
