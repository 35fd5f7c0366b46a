"""The append's cosines and sines on the CPU: the integer steps of the kernel's
own header, compiled for the host, against extended precision."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from exact_io_aware_flashattention_gb300 import _build

SOURCE = r"""
#include "fa_angle.h"
extern "C" void angles(const uint64_t* phase, long n, uint32_t* cos31, uint32_t* sin32, int* quarter, int* negative) {
  for (long i = 0; i < n; ++i) {
    const fa::FixedAngle a = fa::fixed_angle(phase[i]);
    cos31[i] = a.cos31;
    sin32[i] = a.sin32;
    quarter[i] = (int)a.quarter;
    negative[i] = a.negative;
  }
}
"""


@pytest.fixture(scope="module")
def angles(tmp_path_factory):
    where = tmp_path_factory.mktemp("angle")
    src, lib = str(where / "angle.cpp"), str(where / "angle.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", _build.CSRC, src, "-o", lib], check=True)
    call = ctypes.CDLL(lib).angles

    def run(phase):
        n = len(phase)
        out = [np.zeros(n, np.uint32), np.zeros(n, np.uint32), np.zeros(n, np.int32), np.zeros(n, np.int32)]
        call(phase.ctypes.data_as(ctypes.c_void_p), ctypes.c_long(n), *(x.ctypes.data_as(ctypes.c_void_p) for x in out))
        return out
    return run


def phases():
    r = np.random.default_rng(5)
    some = r.integers(0, 2 ** 64, size=400000, dtype=np.uint64)
    small = r.integers(0, 2 ** 64, size=100000, dtype=np.uint64) >> r.integers(0, 64, size=100000, dtype=np.uint64)
    eighths = (np.arange(8, dtype=np.uint64) << np.uint64(61))[:, None] + np.arange(-3, 4).astype(np.int64).view(np.uint64)
    return np.concatenate([some, small, np.uint64(0) - small, eighths.ravel()])


def test_fixed_angles_are_within_2_to_the_minus_29_and_a_half(angles):
    # x and theta are cut (0.39 and 0.5 of 2^-30), and so are the polynomials' products: 0.25 of 2^-30, a unit of 2^-32, for the
    # square, the last product and the cosine's last shift each, with factors of 0.8, 0.5 and 1 at most: less than 2^0.5.
    phase = phases()
    c, s, quarter, negative = angles(phase)
    off = (phase - (quarter.astype(np.uint64) << np.uint64(62))).view(np.int64)            # to the quarter turn, exactly
    assert (np.abs(off.astype(np.float64)) <= 2.0 ** 61).all() and np.array_equal(negative != 0, off < 0)
    theta = np.abs(off.astype(np.longdouble)) * np.longdouble(2) ** -63 * np.longdouble("3.14159265358979323846264338327950288")
    assert np.abs(s.astype(np.longdouble) * np.longdouble(2) ** -32 - np.sin(theta)).max() <= 2.0 ** -29.5
    assert np.abs(c.astype(np.longdouble) * np.longdouble(2) ** -31 - np.cos(theta)).max() <= 2.0 ** -29.5


def test_quarter_turns_are_exact(angles):
    c, s, quarter, negative = angles(np.arange(4, dtype=np.uint64) << np.uint64(62))
    assert (c == 2 ** 31).all() and not s.any() and quarter.tolist() == [0, 1, 2, 3] and not negative.any()
