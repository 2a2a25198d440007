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


def sums(shim, z, top, T, per, unit):
    """Rows [threads, n] of one thread's logits each: their sums in floats."""
    shim.cut_sum.restype = ctypes.c_uint64
    return [shim.cut_sum(at(r), len(r), ctypes.c_float(top), ctypes.c_float(T), per, unit) for r in map(f32, z)]


def check_sums(shim, z, top, T, per):
    """Every thread's sum against the weights' own errors and the sums'."""
    shim.cut_pair_error.restype = shim.cut_sum_error.restype = ctypes.c_float
    shim.cut_sum_error.argtypes = [ctypes.c_float, ctypes.c_int, ctypes.c_int]
    want = exact(f32(z).reshape(-1), top, T).reshape(np.shape(z)).sum(1)
    unit = shim.cut_unit_of(ctypes.c_float(float(want.max()) + 1.0))
    got = np.array(sums(shim, z, top, T, per, unit), np.uint64).astype(np.longdouble) * np.longdouble(2.0) ** -unit
    # (the constant behind sum_error is for all threads of 8 CTAs: 1.5 units each here)
    bound = [shim.cut_pair_error() * float(x) + (shim.cut_sum_error(float(x) * 2.0 ** unit, z.shape[1], unit) - 32768 + 2) * 2.0 ** -unit
             for x in want]
    off = np.abs(got - want).astype(np.float64)
    assert (off <= bound).all(), float((off / bound).max())
    return float((off / want.astype(np.float64)).max())


@pytest.mark.parametrize("per", (4, 8))
def test_sums_in_floats_keep_their_bound(shim, per):
    rng = np.random.default_rng(3)
    for T, offset in ((1.0, 0.0), (0.7, 8.0), (1.3, -40.0), (0.05, 30.0), (2.0, 1000.0)):
        top = np.float32(offset)
        for n in (8, 64, 512):
            for sigma in (0.1, 1.0, 4.0, 12.0):
                z = np.minimum(f32(offset - np.abs(rng.normal(size=(40, n)) * sigma * T)), top)
                check_sums(shim, z, top, T, per)


@pytest.mark.parametrize("per", (4, 8))
def test_sums_in_floats_of_few_and_of_equal_weights(shim, per):
    """A single weight's error counts whole, and equal ones' errors all the same way:
    of weights too small for the first sum, too."""
    rng = np.random.default_rng(4)
    worst = 0.0
    for T, offset in ((1.0, 0.0), (0.7, 7.3), (1.3, -90.0), (0.9, 400.0)):
        top = np.float32(offset)
        z = f32(np.full((20000, 8), offset - 200.0 * T))
        z[:, 3] = np.minimum(f32(offset - rng.uniform(0, 3, 20000) * T), top)
        worst = max(worst, check_sums(shim, z, top, T, per))
        for below in (0.37, 3.0, 9.0, 15.9, 16.6, 17.3, 22.0, 28.0):
            for first in (0.0, 5.0):
                z = f32(np.full((20, 512), offset - below * T) - rng.uniform(0, 0.01, (20, 1)) * T)
                z[:, 7] = offset - first * T
                check_sums(shim, np.minimum(z, top), top, T, per)
    assert worst > 2.0 ** -33  # as single weights are off by
