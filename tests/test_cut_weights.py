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
