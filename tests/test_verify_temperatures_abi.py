"""Host validation of sv_verify_args.temperatures (CPU only: no call here reaches the
GPU)."""
import ctypes

import pytest

from speculative_decoding_verification_24_gb300 import binding
from speculative_decoding_verification_24_gb300.build import build

FAKE = 0x10000  # never dereferenced: every call below fails validation first


def args(**changes):
    a = binding.sv_verify_args()
    a.target_logits = a.draft_logits = a.draft_tokens = a.out_tokens = a.out_n_accepted = FAKE
    a.B, a.K, a.V, a.dtype, a.mode, a.temperature = 2, 3, 100, binding.SV_F32, binding.SV_SAMPLE, 1.0
    for name, value in changes.items():
        setattr(a, name, value)
    return a


@pytest.mark.parametrize("changes,code", [
    (dict(temperatures=FAKE + 2), 9),
    (dict(temperature=float("nan")), 4),
    # with temperatures the number is not looked at
    (dict(temperature=float("nan"), temperatures=FAKE, out_tokens=FAKE + 2), 9),
    (dict(temperature=0.0, temperatures=FAKE, cluster_size=3), 10),
])
def test_validation(changes, code):
    build()
    assert binding.library().spec_verify_ex(ctypes.byref(args(**changes))) == code
