"""Host validation of the operators that cut rows of logits (CPU only: no call
here reaches the GPU) and the binding's checks of its tensors."""
import ctypes

import pytest
import torch

from speculative_decoding_verification_24_gb300 import binding, spec_sample, spec_truncate_logits
from speculative_decoding_verification_24_gb300.build import build

FAKE = 0x10000  # never dereferenced: every call below fails validation first
NULL, SHAPE, DTYPE, TEMPERATURE, ALIGN, CONFIG = 1, 2, 3, 4, 9, 10


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.library()


def cut(**changes):
    c = binding.sv_logits_cut()
    c.logits = FAKE
    c.dtype, c.B, c.R, c.V = binding.SV_F32, 2, 3, 100
    c.seq_stride, c.row_stride = 300, 100
    c.temperature, c.top_p = 1.0, 1.0
    for name, value in changes.items():
        setattr(c, name, value)
    return c


nan, inf = float("nan"), float("inf")


@pytest.mark.parametrize("changes,code", [
    (dict(logits=None), NULL), (dict(dtype=2), DTYPE), (dict(dtype=9), DTYPE),
    (dict(B=0), SHAPE), (dict(R=0), SHAPE), (dict(V=1), SHAPE), (dict(V=2 ** 18 + 1), SHAPE), (dict(B=2 ** 20, R=2 ** 9), SHAPE),
    (dict(seq_stride=-1), SHAPE), (dict(row_stride=-100), SHAPE), (dict(seq_stride=2 ** 41), SHAPE),
    (dict(temperature=-1.0), TEMPERATURE), (dict(temperature=nan), TEMPERATURE), (dict(temperature=inf), TEMPERATURE),
    (dict(temperature=1e-30), TEMPERATURE),
    (dict(top_k=-1), CONFIG), (dict(top_p=-0.1), CONFIG), (dict(top_p=1.1), CONFIG), (dict(top_p=nan), CONFIG),
    (dict(min_p=-0.1), CONFIG), (dict(min_p=1.5), CONFIG), (dict(min_p=nan), CONFIG),
    (dict(logits=FAKE + 2), ALIGN), (dict(logits=FAKE + 1, dtype=1), ALIGN), (dict(temperatures=FAKE + 2), ALIGN),
    (dict(top_ks=FAKE + 1), ALIGN), (dict(top_ps=FAKE + 2), ALIGN), (dict(min_ps=FAKE + 3), ALIGN), (dict(status_word=FAKE + 1), ALIGN),
])
def test_cut_validation(lib, changes, code):
    c = cut(**changes)
    assert lib.spec_sample(ctypes.byref(c), FAKE, FAKE, None) == code
    assert lib.spec_truncate_logits(ctypes.byref(c), FAKE, 300, 100, None) == code


def test_own_arguments(lib):
    c = cut()
    assert lib.spec_sample(None, FAKE, FAKE, None) == NULL
    assert lib.spec_sample(ctypes.byref(c), None, FAKE, None) == NULL
    assert lib.spec_sample(ctypes.byref(c), FAKE, None, None) == NULL
    assert lib.spec_sample(ctypes.byref(c), FAKE + 2, FAKE, None) == ALIGN
    assert lib.spec_sample(ctypes.byref(c), FAKE, FAKE, FAKE + 1) == ALIGN
    assert lib.spec_truncate_logits(None, FAKE, 300, 100, None) == NULL
    assert lib.spec_truncate_logits(ctypes.byref(c), None, 300, 100, None) == NULL
    assert lib.spec_truncate_logits(ctypes.byref(c), FAKE + 2, 300, 100, None) == ALIGN
    assert lib.spec_truncate_logits(ctypes.byref(c), FAKE, 300, 100, FAKE + 2) == ALIGN
    # outputs whose rows share memory
    for seq, row in ((300, 99), (299, 100), (0, 100), (300, 0), (100, 150), (-1, 100)):
        assert lib.spec_truncate_logits(ctypes.byref(c), FAKE, seq, row, None) == SHAPE


def test_binding_refuses_cpu_tensors():
    z = torch.zeros(2, 10)
    with pytest.raises(ValueError):
        spec_sample(z, torch.zeros(2))
    with pytest.raises(ValueError):
        spec_truncate_logits(z)
