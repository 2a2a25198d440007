"""The weights by which tokens are drawn and cut (csrc/cut_weights.cuh), compiled
for the host, against longer arithmetic."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "speculative_decoding_verification_24_gb300", "csrc")


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("cut") / "shim.so")
    # (no contraction: a product and a sum are one rounding only where the source says so)
    subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off", "-shared", "-fPIC", "-I", CSRC,
                    os.path.join(HERE, "cut_weights_shim.cpp"), "-o", so], check=True)
    return ctypes.CDLL(so)


def f32(x):
    return np.ascontiguousarray(x, np.float32)


def at(a):
    return a.ctypes.data_as(ctypes.c_void_p)


def weights(shim, z, top, T):
    out = np.empty(len(z), np.uint64)
    shim.cut_weights(at(z), len(z), ctypes.c_float(top), ctypes.c_float(T), at(out))
    return out


def exact(z, top, T):
    """exp((z - top) / T) with 64 bits of mantissa or more."""
    assert np.finfo(np.longdouble).nmant >= 63
    d = (z.astype(np.longdouble) - np.longdouble(top)) / np.longdouble(np.float32(T))
    return np.exp(d)


def test_a_weight_is_right_to_2_40(shim):
    """Of itself, and 2 units: the units' own rounding is half of one, that of what
    the two float parts are rounded to (each to whole units) as much again."""
    unit = np.longdouble(2.0) ** -shim.cut_unit()
    rng = np.random.default_rng(1)
    for T in (1.0, 0.7, 1.3, 0.05, 3.0, 2.0 ** -20, 1e6):
        for offset in (0.0, 5.0, 300.0):
            top = np.float32(offset * T)
            z = f32(top - rng.exponential(6.0, 40000) * T)
            z = z[z <= top]
            want = exact(z, top, T)
            off = np.abs(weights(shim, z, top, T).astype(np.longdouble) * unit - want)
            assert (off <= 2.0 ** -40 * want + 2 * unit).all(), (T, offset, float((off / (2.0 ** -40 * want + 2 * unit)).max()))
            assert weights(shim, f32([top]), top, T)[0] == 2 ** shim.cut_unit()


def test_weights_in_every_unit(shim):
    """Half a unit, and what the parts are rounded to, 2 times 2^-44 of itself, beside
    the series' 2^-40."""
    rng = np.random.default_rng(2)
    for unit in range(44, 63):
        for T in (1.0, 0.37, 1e-6):
            z = f32(-np.concatenate([rng.exponential(6.0, 5000), rng.uniform(0, 50, 5000), [0.0, 43.0, 200.0, np.inf]]) * T)
            want, out = exact(z, 0.0, T), np.empty(len(z), np.uint64)
            shim.cut_weights_in(at(z), len(z), ctypes.c_float(0.0), ctypes.c_float(T), unit, at(out))
            one = np.longdouble(2.0) ** -unit
            off = np.abs(out.astype(np.longdouble) * one - want)
            bound = (2.0 ** -40 + 2.0 ** -43) * want + 0.5001 * one
            assert (off <= bound).all(), (unit, T, float((off / bound).max()))
            assert out[-4] == 2 ** unit and out[-1] == 0


def test_the_unit_leaves_room_for_the_sum(shim):
    shim.cut_unit_of.argtypes = [ctypes.c_float]
    for sum_ in (0.5, 0.99999, 1.0, 1.5, 1.9999999, 2.0, 3.0, 4.0, 1000.0, 2.0 ** 17, 262143.0, 2.0 ** 18, 2.0 ** 18 * 1.0001):
        unit = shim.cut_unit_of(sum_)
        assert np.float32(sum_).astype(np.float64) * 2.0 ** unit < 2.0 ** 63 and unit <= 62
        assert unit == 62 or np.float64(np.float32(sum_)) * 2.0 ** unit >= 2.0 ** 62
    # what the kernel adds up beforehand is right to 2^-15, and taken as 2^-13 more
    assert shim.cut_unit_of(2.0 ** 18 * (1 + 2.0 ** -13)) == 44
