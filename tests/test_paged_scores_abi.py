"""Host validation of the paged attention's score_cap and bias_slopes (CPU only:
no call here reaches the GPU)."""
import ctypes

import pytest

from speculative_decoding_verification_24_gb300 import binding
from speculative_decoding_verification_24_gb300.build import build
from test_paged_abi import ALIGN, CONFIG, FAKE, attention_args


@pytest.mark.parametrize("changes,code", [
    (dict(score_cap=-1.0), CONFIG), (dict(score_cap=float("nan")), CONFIG), (dict(score_cap=float("inf")), CONFIG),
    (dict(score_cap=5000.0), CONFIG), (dict(score_cap=1e-4), CONFIG), (dict(score_cap=0.01, scale=1e37), CONFIG),
    (dict(bias_slopes=FAKE + 2), ALIGN),
])
def test_refused(changes, code):
    build()
    assert binding.library().spec_paged_attention(ctypes.byref(attention_args(**changes))) == code


@pytest.mark.parametrize("scale,cap", [(2.0 ** -61, 1.0), (2.0 ** 61, 1.0), (2.0 ** -50, 4096.0), (2.0 ** 52, 2.0 ** -10)])
def test_a_scale_too_far_from_the_cap(scale, cap):
    """Neither it nor its square is to be 0 or infinite."""
    build()
    call = binding.library().spec_paged_attention
    assert call(ctypes.byref(attention_args(score_cap=cap, scale=scale))) == CONFIG
