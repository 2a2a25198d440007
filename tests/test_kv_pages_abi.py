"""Host validation of spec_kv_pages (CPU only: no call here reaches the GPU) and
the binding's checks of its tensors."""
import ctypes

import pytest
import torch

from speculative_decoding_verification_24_gb300 import binding, spec_kv_pages
from speculative_decoding_verification_24_gb300.build import build

FAKE = 0x10000  # never dereferenced: every call below fails validation first
NULL, SHAPE, ALIGN = 1, 2, 9


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.library()


def args(**changes):
    a = binding.sv_kv_pages_args()
    a.page_table = a.held = a.free_pages = a.n_free = a.ctx_lens = a.cu_new = a.slots = a.positions = FAKE
    a.page_table_stride = a.max_pages = 8
    a.n_pages, a.page_size, a.B, a.T = 40, 16, 3, 7
    for name, value in changes.items():
        setattr(a, name, value)
    return a


@pytest.mark.parametrize("changes,code", [
    *((dict([(n, None)]), NULL) for n in ("page_table", "held", "free_pages", "n_free", "ctx_lens", "cu_new")),
    (dict(B=0), SHAPE), (dict(B=8193), SHAPE), (dict(max_pages=0), SHAPE), (dict(page_table_stride=7), SHAPE),
    (dict(n_pages=0), SHAPE), (dict(n_pages=2 ** 31 - 1), SHAPE), (dict(page_size=4), SHAPE), (dict(page_size=20), SHAPE),
    (dict(page_size=65544), SHAPE), (dict(T=-1), SHAPE), (dict(max_pages=2 ** 27, page_table_stride=2 ** 27), SHAPE),
    *((dict([(n, FAKE + 2)]), ALIGN) for n in ("page_table", "held", "free_pages", "n_free", "ctx_lens", "cu_new", "positions", "status_word")),
    (dict(slots=FAKE + 4), ALIGN),
])
def test_validation(lib, changes, code):
    assert lib.spec_kv_pages(ctypes.byref(args(**changes))) == code


def test_null_and_cpu_tensors(lib):
    assert lib.spec_kv_pages(None) == NULL
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        spec_kv_pages(i(2, 4), i(2), i(9), i(1), i(2), i(3), 16)
