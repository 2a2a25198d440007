"""Host validation of the paged cache's entry points (CPU only: no call here
reaches the GPU) and the binding's checks of its tensors."""
import ctypes

import pytest
import torch

from speculative_decoding_verification_24_gb300 import binding
from speculative_decoding_verification_24_gb300.build import build

FAKE = 0x10000  # never dereferenced: every call below fails validation first
NULL, SHAPE, DTYPE, WORKSPACE, ALIGN, CONFIG = 1, 2, 3, 5, 9, 10


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.library()


def put(struct, changes):
    for name, value in changes.items():
        setattr(struct, name, value)
    return struct


def cache(**changes):
    c = binding.sv_kv_cache()
    c.k = c.v = c.page_table = c.ctx_lens = FAKE
    c.dtype, c.n_pages, c.page_size, c.Hkv, c.D, c.B, c.max_pages = binding.SV_BF16, 10, 16, 2, 128, 3, 4
    c.k_page_stride = c.v_page_stride = 16 * 2 * 128
    c.k_token_stride = c.v_token_stride = 2 * 128
    c.k_head_stride = c.v_head_stride = 128
    c.page_table_stride = 4
    return put(c, changes)


FREQ = (ctypes.c_double * 64)(*([0.5] * 64))


def append_args(cache_changes=None, **changes):
    a = binding.sv_kv_append_args()
    a.cache = cache(**(cache_changes or {}))
    a.cu_new = a.k = a.v = a.q = a.q_out = FAKE
    a.T, a.Hq = 5, 8
    a.k_token_stride = a.v_token_stride = a.q_token_stride = a.q_out_token_stride = 2048
    a.k_head_stride = a.v_head_stride = a.q_head_stride = a.q_out_head_stride = 128
    a.inv_freq, a.rotary = ctypes.addressof(FREQ), 128
    return put(a, changes)


def attention_args(cache_changes=None, **changes):
    a = binding.sv_paged_attention_args()
    a.cache = cache(**(cache_changes or {}))
    a.cu_new = a.q = a.out = a.workspace = FAKE
    a.T, a.Hq, a.scale, a.workspace_bytes = 5, 8, 0.1, 1 << 30
    a.q_token_stride = a.out_token_stride = 1024
    a.q_head_stride = a.out_head_stride = 128
    return put(a, changes)


BAD_CACHES = [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(page_table=None), NULL), (dict(ctx_lens=None), NULL),
    (dict(dtype=0), DTYPE), (dict(dtype=7), DTYPE),
    (dict(n_pages=0), SHAPE), (dict(n_pages=2 ** 31 - 1), SHAPE), (dict(page_size=0), SHAPE), (dict(page_size=12), SHAPE),
    (dict(page_size=65544), SHAPE), (dict(Hkv=0), SHAPE), (dict(D=96), SHAPE), (dict(D=256), SHAPE), (dict(B=0), SHAPE),
    (dict(max_pages=0), SHAPE), (dict(page_table_stride=3), SHAPE),
    (dict(max_pages=1 << 28, page_table_stride=1 << 28), SHAPE),  # slots past int32
    (dict(k=FAKE + 8), ALIGN), (dict(v=FAKE + 2), ALIGN), (dict(page_table=FAKE + 2), ALIGN), (dict(ctx_lens=FAKE + 1), ALIGN),
    (dict(k_page_stride=0), SHAPE), (dict(v_token_stride=0), SHAPE), (dict(v_head_stride=0), SHAPE),
    (dict(k_page_stride=4100), ALIGN), (dict(v_token_stride=257), ALIGN), (dict(k_head_stride=-128), ALIGN),
]


@pytest.mark.parametrize("changes,code", BAD_CACHES)
def test_cache_validation(lib, changes, code):
    assert lib.spec_kv_append(ctypes.byref(append_args(changes))) == code
    assert lib.spec_paged_attention(ctypes.byref(attention_args(changes))) == code
    c = cache(**changes)
    assert lib.spec_kv_commit(ctypes.byref(c), FAKE, FAKE, 8, FAKE, FAKE, None, None) == code


@pytest.mark.parametrize("changes,code", [
    (dict(cu_new=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(q_out=None), NULL), (dict(inv_freq=None), NULL),
    (dict(T=-1), SHAPE), (dict(Hq=0), SHAPE), (dict(rotary=24), SHAPE), (dict(rotary=-16), SHAPE), (dict(rotary=144), SHAPE),
    (dict(tree_parents=FAKE, N=0), SHAPE), (dict(tree_parents=FAKE, N=33), SHAPE),
    (dict(cu_new=FAKE + 2), ALIGN), (dict(k=FAKE + 8), ALIGN), (dict(q=FAKE + 4), ALIGN), (dict(q_out=FAKE + 2), ALIGN),
    (dict(positions=FAKE + 1), ALIGN), (dict(status_word=FAKE + 2), ALIGN), (dict(tree_parents=FAKE + 2, N=8), ALIGN),
    (dict(k_token_stride=2049), ALIGN), (dict(q_out_head_stride=129), ALIGN), (dict(v_head_stride=-128), ALIGN),
])
def test_append_validation(lib, changes, code):
    assert lib.spec_kv_append(ctypes.byref(append_args(**changes))) == code


def test_append_refuses_frequencies_that_are_not_finite(lib):
    for bad in (float("inf"), float("nan")):
        f = (ctypes.c_double * 64)(*([0.5] * 63 + [bad]))
        assert lib.spec_kv_append(ctypes.byref(append_args(inv_freq=ctypes.addressof(f)))) == CONFIG


@pytest.mark.parametrize("changes,code", [
    (dict(cu_new=None), NULL), (dict(q=None), NULL), (dict(out=None), NULL),
    (dict(T=-1), SHAPE), (dict(Hq=0), SHAPE), (dict(Hq=7), SHAPE), (dict(Hq=258), SHAPE),
    (dict(tree_parents=FAKE, N=33), SHAPE),
    (dict(scale=0.0), CONFIG), (dict(scale=-1.0), CONFIG), (dict(scale=float("nan")), CONFIG), (dict(scale=float("inf")), CONFIG),
    (dict(scale=3e38), CONFIG), (dict(flags=1), CONFIG),
    (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=1024), WORKSPACE),
    (dict(workspace=FAKE + 128), ALIGN), (dict(q=FAKE + 8), ALIGN), (dict(out=FAKE + 8), ALIGN), (dict(out_lse=FAKE + 2), ALIGN),
    (dict(cu_new=FAKE + 1), ALIGN), (dict(q_token_stride=1028), ALIGN), (dict(out_head_stride=100), ALIGN),
])
def test_attention_validation(lib, changes, code):
    assert lib.spec_paged_attention(ctypes.byref(attention_args(**changes))) == code


@pytest.mark.parametrize("args,code", [
    ((None, FAKE, 8, FAKE, FAKE), NULL), ((FAKE, FAKE, 8, None, FAKE), NULL), ((FAKE, FAKE, 8, FAKE, None), NULL),
    ((FAKE, FAKE, 0, FAKE, FAKE), SHAPE), ((FAKE, FAKE, 33, FAKE, FAKE), SHAPE),
    ((FAKE + 2, None, 0, None, FAKE), ALIGN), ((FAKE, FAKE, 8, FAKE + 1, FAKE), ALIGN), ((FAKE, None, 0, None, FAKE + 2), ALIGN),
])
def test_commit_validation(lib, args, code):
    n, parents, N, last, out = args
    assert lib.spec_kv_commit(ctypes.byref(cache()), n, parents, N, last, out, None, None) == code


def test_null_structs(lib):
    assert lib.spec_kv_append(None) == NULL
    assert lib.spec_paged_attention(None) == NULL
    assert lib.spec_kv_commit(None, FAKE, None, 0, None, FAKE, None, None) == NULL


def test_workspace_bytes(lib):
    f = lib.spec_paged_attention_workspace_bytes
    # 2 * 160 pieces of (m, l) and D floats per row; rows: all packed ones up
    # to one tile of 128, in steps of 32, then a pair of tiles
    assert f(1, 8, 2, 128) == 1024 + 320 * 32 * (8 + 512)
    assert f(9, 32, 8, 64) == 1024 + 320 * 64 * (8 + 256)
    assert f(32, 32, 8, 128) == 1024 + 320 * 128 * (8 + 512)
    assert f(33, 32, 8, 128) == f(100000, 32, 8, 128) == 1024 + 320 * 256 * (8 + 512)
    assert f(0, 8, 2, 128) == 1024
    assert f(-1, 8, 2, 128) == f(1, 7, 2, 128) == f(1, 129, 1, 128) == f(1, 8, 2, 96) == f(1, 0, 1, 64) == 0


def test_binding_checks_its_tensors(lib):
    from speculative_decoding_verification_24_gb300 import spec_kv_append, spec_kv_commit, spec_paged_attention
    cache = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    ints = torch.zeros(3, dtype=torch.int32)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    for call in (lambda: spec_paged_attention(q, cache, cache, ints.view(1, 3), ints[:1], ints[:2]),
                 lambda: spec_kv_append(q[:, :2], q[:, :2], cache, cache, ints.view(1, 3), ints[:1], ints[:2]),
                 lambda: spec_kv_commit(cache, cache, ints.view(1, 3), ints[:1], ints[:1])):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_binding_refuses_an_output_of_queries_that_are_not_given():
    from speculative_decoding_verification_24_gb300 import spec_kv_append
    cache, ints = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="q_out is given without q"):
        spec_kv_append(k, k, cache, cache, ints.view(1, 3), ints[:1], ints[:2], q_out=k)


def test_binding_checks_status_and_plain_tensors():
    one = torch.zeros(1, dtype=torch.int32)
    assert binding._status(None, 0) == 0
    for bad in (one.float(), one.long(), one.to(torch.uint8)):
        with pytest.raises(TypeError, match="status_word"):
            binding._status(bad, 0)
    with pytest.raises(ValueError, match="no element"):
        binding._status(one[:0], 0)
    for good in (one, one.view(torch.uint32), one.view(()), torch.zeros(4, dtype=torch.int32)):
        with pytest.raises(ValueError, match="CUDA device"):  # of a device that is not the cache's
            binding._status(good, 0)
        assert binding._status(good, -1) == good.data_ptr()
    x = torch.zeros(4, 6)
    with pytest.raises(ValueError, match="workspace must live"):
        binding._plain(x, "workspace", 0)
    with pytest.raises(ValueError, match="out_lse must be contiguous"):
        binding._plain(x.t(), "out_lse", -1)
    assert binding._plain(x, "workspace", -1) == x.data_ptr()


@pytest.mark.parametrize("name", ["out_token_stride", "out_head_stride", "q_token_stride", "q_head_stride"])
def test_attention_refuses_rows_without_places_of_their_own(lib, name):
    assert lib.spec_paged_attention(ctypes.byref(attention_args(**{name: 0}))) == SHAPE
    # one token or head has no next one (no workspace: the next check)
    one = dict(T=1) if "token" in name else dict(Hq=1)
    cache_changes = {} if "token" in name else dict(Hkv=1)
    assert lib.spec_paged_attention(ctypes.byref(attention_args(cache_changes, workspace=None, **one, **{name: 0}))) == WORKSPACE


@pytest.mark.parametrize("name", ["q_out_token_stride", "q_out_head_stride"])
def test_append_refuses_rows_without_places_of_their_own(lib, name):
    assert lib.spec_kv_append(ctypes.byref(append_args(**{name: 0}))) == SHAPE
    one = dict(T=1) if "token" in name else dict(Hq=1)
    bad = (ctypes.c_double * 64)(*([float("nan")] * 64))  # the next check
    assert lib.spec_kv_append(ctypes.byref(append_args(**one, **{name: 0}, inv_freq=ctypes.addressof(bad)))) == CONFIG
    for read in ("k_token_stride", "v_head_stride", "q_token_stride"):
        assert lib.spec_kv_append(ctypes.byref(append_args(**{read: 0}, inv_freq=ctypes.addressof(bad)))) == CONFIG


def test_a_call_on_another_device_makes_it_current(monkeypatch):
    current = [0]

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *exc):
            current[0] = self.before

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    seen = []
    binding._call("f", 1, lambda x: seen.append((x, current[0])) or 0, 5)
    binding._call("f", 0, lambda x: seen.append((x, current[0])) or 0, 6)
    assert seen == [(5, 1), (6, 0)] and current == [0]
    with pytest.raises(binding.SpecVerifyError, match="f"):
        binding._call("f", 1, lambda: SHAPE)
    assert current == [0]
