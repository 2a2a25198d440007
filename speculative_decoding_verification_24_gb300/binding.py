"""Thin ctypes binding of libspecverify (argument marshalling only).

Every function takes torch tensors that already live on the current CUDA
device, passes their data pointers and the current torch stream to the C ABI
declared in include/specverify.h, and raises SpecVerifyError on a non-OK
status. All of the verify arithmetic runs in the library's CUDA kernels; this
module computes nothing. Missing outputs are allocated with torch.empty, under
the stream of the call. Where that is not the current stream (stream=), the
caller orders it after the work that makes the inputs, and what reads the
outputs after it.
"""
from __future__ import annotations

import ctypes
import os
import struct as _struct
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libspecverify.so")
DEBUG_LIB_PATH = os.path.join(_PKG, "libspecverify_debug.so")

SV_F32, SV_BF16, SV_F16 = 0, 1, 2
SV_GREEDY, SV_SAMPLE = 0, 1

SV_FLAG_BAD_TOKEN = 1
SV_FLAG_BAD_ROW = 2
SV_FLAG_RESIDUAL_FALLBACK = 4
SV_FLAG_DRAW_EDGE = 8
SV_FLAG_BAD_MODE = 16
SV_FLAG_TIMEOUT = 32
SV_FLAG_BAD_LENGTH = 64
SV_FLAG_BAD_TREE = 128
SV_FLAG_DEBUG_BOUNDS = 256
SV_FLAG_BAD_PAGE = 512
SV_ARG_OVERLAP_PREVIOUS = 1
SV_ARG_TEST_WAIT_TIMEOUT = 0x80000000
SV_ARG_TEST_DEBUG_SHRINK = 0x40000000
SV_ERR_SCRATCH_LIMIT = 12
SV_LMHEAD_SCRATCH_BYTES = 32 << 20  # include/specverify.h
SV_PAGED_WORKSPACE_HEAD = 1024  # include/specverify.h

STATUS_NAMES = {
    0: "SV_OK", 1: "SV_ERR_NULL", 2: "SV_ERR_SHAPE", 3: "SV_ERR_DTYPE", 4: "SV_ERR_TEMPERATURE",
    5: "SV_ERR_WORKSPACE", 6: "SV_ERR_ARCH", 7: "SV_ERR_CUDA", 8: "SV_ERR_MODE",
    9: "SV_ERR_ALIGN", 10: "SV_ERR_CONFIG", 11: "SV_ERR_NOT_IMPLEMENTED",
}


class SpecVerifyError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: {STATUS_NAMES.get(status, status)} ({sv_status_string(status)})"
        if status == 7:
            msg += f"; cuda error {_load().sv_last_cuda_error()}"
        super().__init__(msg)


class sv_verify_args(ctypes.Structure):
    """Mirror of sv_verify_args in include/specverify.h."""
    _fields_ = [
        ("target_logits", ctypes.c_void_p),
        ("draft_logits", ctypes.c_void_p),
        ("draft_tokens", ctypes.c_void_p),
        ("B", ctypes.c_int),
        ("K", ctypes.c_int),
        ("V", ctypes.c_int),
        ("dtype", ctypes.c_int),
        ("temperature", ctypes.c_float),
        ("mode", ctypes.c_int),
        ("modes", ctypes.c_void_p),
        ("seed", ctypes.c_uint64),
        ("seq_ids", ctypes.c_void_p),
        ("out_tokens", ctypes.c_void_p),
        ("out_n_accepted", ctypes.c_void_p),
        ("out_p_target", ctypes.c_void_p),
        ("out_p_draft", ctypes.c_void_p),
        ("out_residual_mass", ctypes.c_void_p),
        ("status_word", ctypes.c_void_p),
        ("cluster_size", ctypes.c_int),
        ("stream", ctypes.c_void_p),
        ("flags", ctypes.c_uint32),
        ("draft_lens", ctypes.c_void_p),
        ("out_draw_edges", ctypes.c_void_p),
        ("seqs_per_cluster", ctypes.c_int),
    ]


class sv_verify_plan(ctypes.Structure):
    """Mirror of sv_verify_plan in include/specverify.h."""
    _fields_ = [
        ("grouped", ctypes.c_int),
        ("clusters", ctypes.c_int),
        ("cluster_size", ctypes.c_int),
        ("max_seqs_per_cluster", ctypes.c_int),
    ]


class sv_kv_cache(ctypes.Structure):
    """Mirror of sv_kv_cache in include/specverify.h."""
    _fields_ = [
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("dtype", ctypes.c_int),
        ("n_pages", ctypes.c_int),
        ("page_size", ctypes.c_int),
        ("Hkv", ctypes.c_int),
        ("D", ctypes.c_int),
        ("B", ctypes.c_int),
        ("k_page_stride", ctypes.c_int64),
        ("k_token_stride", ctypes.c_int64),
        ("k_head_stride", ctypes.c_int64),
        ("v_page_stride", ctypes.c_int64),
        ("v_token_stride", ctypes.c_int64),
        ("v_head_stride", ctypes.c_int64),
        ("page_table", ctypes.c_void_p),
        ("page_table_stride", ctypes.c_int64),
        ("max_pages", ctypes.c_int),
        ("ctx_lens", ctypes.c_void_p),
    ]


class sv_kv_append_args(ctypes.Structure):
    """Mirror of sv_kv_append_args in include/specverify.h."""
    _fields_ = [
        ("cache", sv_kv_cache),
        ("cu_new", ctypes.c_void_p),
        ("T", ctypes.c_int),
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("k_token_stride", ctypes.c_int64),
        ("k_head_stride", ctypes.c_int64),
        ("v_token_stride", ctypes.c_int64),
        ("v_head_stride", ctypes.c_int64),
        ("Hq", ctypes.c_int),
        ("q", ctypes.c_void_p),
        ("q_out", ctypes.c_void_p),
        ("q_token_stride", ctypes.c_int64),
        ("q_head_stride", ctypes.c_int64),
        ("q_out_token_stride", ctypes.c_int64),
        ("q_out_head_stride", ctypes.c_int64),
        ("inv_freq", ctypes.c_void_p),
        ("rotary", ctypes.c_int),
        ("interleaved", ctypes.c_int),
        ("tree_parents", ctypes.c_void_p),
        ("N", ctypes.c_int),
        ("positions", ctypes.c_void_p),
        ("status_word", ctypes.c_void_p),
        ("stream", ctypes.c_void_p),
    ]


class sv_paged_attention_args(ctypes.Structure):
    """Mirror of sv_paged_attention_args in include/specverify.h."""
    _fields_ = [
        ("cache", sv_kv_cache),
        ("cu_new", ctypes.c_void_p),
        ("T", ctypes.c_int),
        ("Hq", ctypes.c_int),
        ("q", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("q_token_stride", ctypes.c_int64),
        ("q_head_stride", ctypes.c_int64),
        ("out_token_stride", ctypes.c_int64),
        ("out_head_stride", ctypes.c_int64),
        ("out_lse", ctypes.c_void_p),
        ("scale", ctypes.c_float),
        ("tree_parents", ctypes.c_void_p),
        ("N", ctypes.c_int),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("status_word", ctypes.c_void_p),
        ("flags", ctypes.c_uint32),
        ("stream", ctypes.c_void_p),
    ]


_lock = threading.Lock()
_lib = None

# (name, restype, argtypes) of every symbol the header declares.
P = ctypes.c_void_p
I = ctypes.c_int
SIGNATURES = [
    ("spec_verify", I, [P, P, P, I, I, I, I, ctypes.c_float, I, ctypes.c_uint64, P, P, P]),
    ("spec_verify_ex", I, [ctypes.POINTER(sv_verify_args)]),
    ("spec_verify_plan", I, [ctypes.POINTER(sv_verify_args), ctypes.POINTER(sv_verify_plan)]),
    ("spec_verify_lmhead_workspace_bytes", ctypes.c_size_t, [I, I, I, I]),
    ("spec_verify_lmhead", I, [P, P, P, P, I, I, I, I, I, ctypes.c_float, I, ctypes.c_uint64, P,
                               ctypes.c_size_t, P, P, P]),
    ("spec_lmhead_logits", I, [P, P, I, I, I, P, P]),
    ("spec_verify_tree", I, [P, I, P, P, I, I, I, P, P, P, P]),
    ("spec_prompt_lookup", I, [P, P, I, I, I, I, P, P, P]),
    ("spec_commit", I, [P, P, I, I, P, P, I, P, P]),
    ("spec_verify_lmhead_noalloc", I, [P, P, P, P, I, I, I, I, I, ctypes.c_float, I,
                                       ctypes.c_uint64, P, P, P]),
    ("spec_kv_append", I, [P]),  # sv_kv_append_args*
    ("spec_paged_attention_workspace_bytes", ctypes.c_size_t, [I, I, I, I]),
    ("spec_paged_attention", I, [P]),  # sv_paged_attention_args*
    ("spec_kv_commit", I, [P, P, P, I, P, P, P, P]),
    ("sv_kv_cache_size", ctypes.c_size_t, []),
    ("sv_kv_append_args_size", ctypes.c_size_t, []),
    ("sv_paged_attention_args_size", ctypes.c_size_t, []),
    ("sv_status_string", ctypes.c_char_p, [I]),
    ("sv_last_cuda_error", I, []),
    ("sv_version", I, []),
    ("sv_verify_args_size", ctypes.c_size_t, []),
]


def load_library(path: str):
    """Load one build of the library (release or debug) and declare the
    signatures of every symbol the header declares; fail loudly when it has
    not been built."""
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it with "
            "`python -c 'import __graft_entry__ as g; g.build()'` (there is no fallback)")
    lib = ctypes.CDLL(path)
    for name, res, args in SIGNATURES:
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if lib.sv_verify_args_size() != ctypes.sizeof(sv_verify_args):
        raise ImportError("sv_verify_args layout differs between the binding and the library")
    for struct in (sv_kv_cache, sv_kv_append_args, sv_paged_attention_args):
        if getattr(lib, struct.__name__ + "_size")() != ctypes.sizeof(struct):
            raise ImportError(f"{struct.__name__} layout differs between the binding and the library")
    return lib


def _load():
    """The in-tree release library, loaded once."""
    global _lib
    with _lock:
        if _lib is None:
            _lib = load_library(LIB_PATH)
    return _lib


def library():
    return _load()


def sv_status_string(status: int) -> str:
    return _load().sv_status_string(int(status)).decode()


def sv_version() -> int:
    return int(_load().sv_version())


def _check(status: int, where: str):
    if status != 0:
        raise SpecVerifyError(int(status), where)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SV_F32
    if t.dtype == torch.bfloat16:
        return SV_BF16
    raise TypeError(f"logits must be float32 or bfloat16, got {t.dtype}")


def _mode_code(mode) -> int:
    if mode in ("greedy", SV_GREEDY):
        return SV_GREEDY
    if mode in ("sample", SV_SAMPLE):
        return SV_SAMPLE
    raise ValueError(f"mode must be 'greedy' or 'sample', got {mode!r}")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("every tensor must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("every tensor must be contiguous")
    return t.data_ptr()


def _stream(stream, device):
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _as_stream(stream, device):
    """The torch stream of a stream or a raw handle. 0 and 1 (cudaStreamLegacy)
    are the default stream, for which ExternalStream would give a new one."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream), device=device) if int(stream) > 1 else torch.cuda.default_stream(device)


def _empty(shape, dtype, device, stream, zero=False):
    """A tensor that a call on `stream` writes. It is allocated under that
    stream: memory of the current one may still be in use by work that is
    enqueued there, and would be handed out again there while this call writes
    it. The current stream, which the caller goes on with, holds it too."""
    make = torch.zeros if zero else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    stream, current = _as_stream(stream, device), torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        t = make(shape, dtype=dtype, device=device)
    if stream != current:
        t.record_stream(current)
    return t


def spec_verify(target_logits, draft_logits, draft_tokens, temperature=1.0, mode="sample", seed=0,
                out_tokens=None, out_n_accepted=None, stream=None):
    """Verify a batch: returns (out_tokens [B, K+1] int32, out_n_accepted [B] int32)."""
    B, K1, V = target_logits.shape
    K = K1 - 1
    dev = target_logits.device
    if out_tokens is None:
        out_tokens = _empty((B, K1), torch.int32, dev, stream)
    if out_n_accepted is None:
        out_n_accepted = _empty((B,), torch.int32, dev, stream)
    with torch.cuda.device(dev):
        st = _load().spec_verify(
            _ptr(target_logits), _ptr(draft_logits), _ptr(draft_tokens), B, K, V,
            _dtype_code(target_logits), float(temperature), _mode_code(mode),
            ctypes.c_uint64(int(seed) & (2**64 - 1)), _ptr(out_tokens), _ptr(out_n_accepted),
            _stream(stream, dev))
    _check(st, "spec_verify")
    return out_tokens, out_n_accepted


def spec_verify_ex(target_logits, draft_logits, draft_tokens, temperature=1.0, modes="sample",
                   seed=0, seq_ids=None, out_tokens=None, out_n_accepted=None, out_p_target=None,
                   out_p_draft=None, out_residual_mass=None, status_word=None, cluster_size=0,
                   stream=None, debug=False, overlap_previous=False, draft_lens=None, flags=0,
                   out_draw_edges=None, lib=None, seqs_per_cluster=0, plan_only=False):
    """Verify with per-sequence modes ([B] int32 tensor, or 'greedy'/'sample'
    for all), explicit Philox sequence ids and optional debug outputs.
    debug=True allocates out_p_target, out_p_draft, out_residual_mass,
    out_draw_edges and status_word. overlap_previous=True sets SV_ARG_OVERLAP_PREVIOUS (the
    inputs are not written by the work just before this call on the stream).
    draft_lens: optional [B] int32 device tensor of per-sequence draft counts.
    lib: a handle from load_library() to call another build of the library
    (the debug build); the release library by default.
    seqs_per_cluster: 0 automatic, 1 one cluster per sequence, 2..8 that many
    sequences per cluster of cluster_size CTAs (calls without overlap).
    plan_only=True: enqueue nothing and return the launch the call would make
    (spec_verify_plan): {"grouped", "clusters", "cluster_size",
    "max_seqs_per_cluster"}.
    Returns a dict of the output tensors."""
    B, K1, V = target_logits.shape
    K = K1 - 1
    dev = target_logits.device
    a = sv_verify_args()
    if out_tokens is None:
        out_tokens = _empty((B, K1), torch.int32, dev, stream)
    if out_n_accepted is None:
        out_n_accepted = _empty((B,), torch.int32, dev, stream)
    if debug:
        if out_p_target is None:
            out_p_target = _empty((B, K), torch.float32, dev, stream)
        if out_p_draft is None:
            out_p_draft = _empty((B, K), torch.float32, dev, stream)
        if out_residual_mass is None:
            out_residual_mass = _empty((B,), torch.float32, dev, stream)
        if status_word is None:
            status_word = _empty((1,), torch.int32, dev, stream, zero=True)
        if out_draw_edges is None:
            out_draw_edges = _empty((B, 2), torch.float32, dev, stream)
    a.target_logits = _ptr(target_logits)
    a.draft_logits = _ptr(draft_logits)
    a.draft_tokens = _ptr(draft_tokens)
    a.B, a.K, a.V = B, K, V
    a.dtype = _dtype_code(target_logits)
    a.temperature = float(temperature)
    if isinstance(modes, torch.Tensor):
        a.mode = SV_SAMPLE
        a.modes = _ptr(modes)
    else:
        a.mode = _mode_code(modes)
        a.modes = None
    a.seed = int(seed) & (2**64 - 1)
    a.seq_ids = _ptr(seq_ids)
    a.out_tokens = _ptr(out_tokens)
    a.out_n_accepted = _ptr(out_n_accepted)
    a.out_p_target = _ptr(out_p_target)
    a.out_p_draft = _ptr(out_p_draft)
    a.out_residual_mass = _ptr(out_residual_mass)
    a.status_word = _ptr(status_word)
    a.cluster_size = int(cluster_size)
    a.flags = (SV_ARG_OVERLAP_PREVIOUS if overlap_previous else 0) | int(flags)
    a.draft_lens = _ptr(draft_lens)
    a.out_draw_edges = _ptr(out_draw_edges)
    a.seqs_per_cluster = int(seqs_per_cluster)
    with torch.cuda.device(dev):
        a.stream = _stream(stream, dev)
        if plan_only:
            plan = sv_verify_plan()
            st = (lib or _load()).spec_verify_plan(ctypes.byref(a), ctypes.byref(plan))
            _check(st, "spec_verify_plan")
            return {"grouped": bool(plan.grouped), "clusters": plan.clusters, "cluster_size": plan.cluster_size,
                    "max_seqs_per_cluster": plan.max_seqs_per_cluster}
        st = (lib or _load()).spec_verify_ex(ctypes.byref(a))
    _check(st, "spec_verify_ex")
    return {"tokens": out_tokens, "n_accepted": out_n_accepted, "p_target": out_p_target,
            "p_draft": out_p_draft, "residual_mass": out_residual_mass,
            "draw_edges": out_draw_edges, "status_word": status_word}


def spec_verify_plan(target_logits, draft_logits, draft_tokens, temperature=1.0, **kw):
    """The launch spec_verify_ex would make for these arguments (nothing is
    enqueued): {"grouped", "clusters", "cluster_size", "max_seqs_per_cluster"}."""
    return spec_verify_ex(target_logits, draft_logits, draft_tokens, temperature, plan_only=True, **kw)


def spec_verify_tree(target_logits, tree_tokens, tree_parents, out_tokens=None, out_n_accepted=None,
                     out_last_node=None, stream=None):
    """Greedy tree verification: target_logits [B, N, V], tree_tokens and
    tree_parents [B, N] int32 (node 0 is the root). Returns (tokens [B, N],
    n_accepted [B], last_node [B])."""
    B, N, V = target_logits.shape
    dev = target_logits.device
    if out_tokens is None:
        out_tokens = _empty((B, N), torch.int32, dev, stream)
    if out_n_accepted is None:
        out_n_accepted = _empty((B,), torch.int32, dev, stream)
    if out_last_node is None:
        out_last_node = _empty((B,), torch.int32, dev, stream)
    with torch.cuda.device(dev):
        st = _load().spec_verify_tree(_ptr(target_logits), _dtype_code(target_logits), _ptr(tree_tokens),
                                      _ptr(tree_parents), B, N, V, _ptr(out_tokens), _ptr(out_n_accepted),
                                      _ptr(out_last_node), _stream(stream, dev))
    _check(st, "spec_verify_tree")
    return out_tokens, out_n_accepted, out_last_node


def spec_prompt_lookup(tokens, lengths, max_ngram=3, n_drafts=5, out_drafts=None, out_n_drafts=None,
                       stream=None):
    """Prompt lookup drafting: tokens [B, L_max] int32, lengths [B] int32
    (device). Returns (drafts [B, n_drafts] -1 padded, n_drafts [B])."""
    B, L_max = tokens.shape
    dev = tokens.device
    if out_drafts is None:
        out_drafts = _empty((B, n_drafts), torch.int32, dev, stream)
    if out_n_drafts is None:
        out_n_drafts = _empty((B,), torch.int32, dev, stream)
    with torch.cuda.device(dev):
        st = _load().spec_prompt_lookup(_ptr(tokens), _ptr(lengths), B, L_max, int(max_ngram),
                                        int(n_drafts), _ptr(out_drafts), _ptr(out_n_drafts),
                                        _stream(stream, dev))
    _check(st, "spec_prompt_lookup")
    return out_drafts, out_n_drafts


def spec_commit(tokens, lengths, out_tokens, n_accepted, out_n_committed=None, stream=None):
    """Append each sequence's accepted drafts and next token to its context
    (tokens [B, L_max], lengths [B], updated in place). Returns the number of
    tokens committed per sequence."""
    B, L_max = tokens.shape
    K = out_tokens.shape[1] - 1
    dev = tokens.device
    if out_n_committed is None:
        out_n_committed = _empty((B,), torch.int32, dev, stream)
    with torch.cuda.device(dev):
        st = _load().spec_commit(_ptr(tokens), _ptr(lengths), B, L_max, _ptr(out_tokens), _ptr(n_accepted), K,
                                 _ptr(out_n_committed), _stream(stream, dev))
    _check(st, "spec_commit")
    return out_n_committed


def spec_lmhead_logits(hidden, W, out=None, stream=None):
    """fp32 logits [M, V] = hidden [M, d] (bf16) . W [d, V] (bf16) on the tensor cores."""
    hidden = hidden.reshape(-1, hidden.shape[-1])
    M, d = hidden.shape
    V = W.shape[1]
    dev = hidden.device
    if out is None:
        out = _empty((M, V), torch.float32, dev, stream)
    with torch.cuda.device(dev):
        st = _load().spec_lmhead_logits(_ptr(hidden), _ptr(W), M, d, V, _ptr(out), _stream(stream, dev))
    _check(st, "spec_lmhead_logits")
    return out


def spec_verify_lmhead_workspace_bytes(B: int, K: int, d: int, V: int) -> int:
    return int(_load().spec_verify_lmhead_workspace_bytes(B, K, d, V))


def spec_verify_lmhead(hidden, W, draft_logits, draft_tokens, temperature=1.0, mode="sample",
                       seed=0, workspace=None, out_tokens=None, out_n_accepted=None, stream=None,
                       lib=None):
    """Fused LM head + verify: hidden [B, K+1, d] bf16, W [d, V] bf16. lib: as
    in spec_verify_ex."""
    B, K1, d = hidden.shape
    K = K1 - 1
    V = W.shape[1]
    dev = hidden.device
    need = spec_verify_lmhead_workspace_bytes(B, K, d, V)
    if workspace is None:
        workspace = _empty((max(need, 1),), torch.uint8, dev, stream)
    if out_tokens is None:
        out_tokens = _empty((B, K1), torch.int32, dev, stream)
    if out_n_accepted is None:
        out_n_accepted = _empty((B,), torch.int32, dev, stream)
    ddt = _dtype_code(draft_logits) if draft_logits is not None else SV_BF16
    with torch.cuda.device(dev):
        st = (lib or _load()).spec_verify_lmhead(
            _ptr(hidden), _ptr(W), _ptr(draft_logits), _ptr(draft_tokens), B, K, d, V, ddt,
            float(temperature), _mode_code(mode), ctypes.c_uint64(int(seed) & (2**64 - 1)),
            _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(out_tokens),
            _ptr(out_n_accepted), _stream(stream, dev))
    _check(st, "spec_verify_lmhead")
    return out_tokens, out_n_accepted


def spec_verify_lmhead_noalloc(hidden, W, draft_logits, draft_tokens, temperature=1.0,
                               mode="sample", seed=0, out_tokens=None, out_n_accepted=None,
                               stream=None):
    """spec_verify_lmhead with its workspace (logits and per-tile partials)
    in the library's own static device scratch (SV_LMHEAD_SCRATCH_BYTES): the
    C call allocates nothing. Calls
    that may overlap on one device race on that scratch; order them."""
    B, K1, d = hidden.shape
    K = K1 - 1
    V = W.shape[1]
    dev = hidden.device
    if out_tokens is None:
        out_tokens = _empty((B, K1), torch.int32, dev, stream)
    if out_n_accepted is None:
        out_n_accepted = _empty((B,), torch.int32, dev, stream)
    ddt = _dtype_code(draft_logits) if draft_logits is not None else SV_BF16
    with torch.cuda.device(dev):
        st = _load().spec_verify_lmhead_noalloc(
            _ptr(hidden), _ptr(W), _ptr(draft_logits), _ptr(draft_tokens), B, K, d, V, ddt,
            float(temperature), _mode_code(mode), ctypes.c_uint64(int(seed) & (2**64 - 1)),
            _ptr(out_tokens), _ptr(out_n_accepted), _stream(stream, dev))
    _check(st, "spec_verify_lmhead_noalloc")
    return out_tokens, out_n_accepted


# ------------------------------------------------------ the paged cache
#
# These calls are short (a few microseconds on the GPU), so their arguments
# are packed in one step instead of field by field.


def _packer(struct):
    """A struct.Struct of the native layout of a ctypes structure, whose
    fields (nested ones in their place) are its arguments in order."""
    codes = {ctypes.c_void_p: "P", ctypes.c_int: "i", ctypes.c_int64: "q", ctypes.c_uint32: "I", ctypes.c_float: "f",
             ctypes.c_size_t: "N"}

    def fields(st):
        return "".join(fields(t) if issubclass(t, ctypes.Structure) else codes[t] for _, t in st._fields_)

    packer = _struct.Struct("@" + fields(struct) + "0q")
    assert packer.size == ctypes.sizeof(struct)
    return packer.pack


_pack_cache, _pack_append, _pack_attention = map(_packer, (sv_kv_cache, sv_kv_append_args, sv_paged_attention_args))
_KV_DTYPES = {torch.bfloat16: SV_BF16, torch.float16: SV_F16}
_I32 = torch.int32


def _rows(t, name, rows, heads, width, dtype, index):
    """Data pointer, strides of the first two dimensions and sizes of them of a
    [rows, heads, width] tensor (any number where None) of any strides but the
    last, on CUDA device `index`."""
    try:
        n, h, w = t.shape
    except ValueError:
        n = h = w = -1
    if w != width or (heads is not None and h != heads) or (rows is not None and n != rows):
        raise ValueError(f"{name} must be [{'T' if rows is None else rows}, {'heads' if heads is None else heads}, {width}], "
                         f"got {list(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype} like the cache, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must live on the cache's CUDA device")
    st, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return t.data_ptr(), st, sh, n, h


def _int32(t, name, index, *shape):
    """Data pointer of a contiguous int32 tensor of that shape on CUDA device
    `index`."""
    if t.dtype is not _I32:
        raise TypeError(f"{name} must be int32, got {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {list(shape)}, got {list(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} must live on the cache's CUDA device")
    return t.data_ptr()


def _plain(t, name, index):
    """Data pointer of a contiguous tensor on CUDA device `index`."""
    if t.get_device() != index:
        raise ValueError(f"{name} must live on the cache's CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _status(t, index):
    if t is None:
        return 0
    if t.dtype is not _I32 and t.dtype is not torch.uint32:
        raise TypeError(f"status_word must be int32 or uint32, got {t.dtype}")
    if t.numel() == 0:
        raise ValueError("status_word has no element")
    return _plain(t, "status_word", index)


def _cache_fields(k_cache, v_cache, page_table, ctx_lens):
    """The fields of sv_kv_cache from k_cache and v_cache [n_pages, page_size,
    Hkv, D] (any strides but the last), page_table [B, max_pages] and ctx_lens
    [B], and the CUDA device they are on."""
    index = k_cache.get_device()
    if index < 0 or v_cache.get_device() != index or page_table.get_device() != index:
        raise ValueError("k_cache, v_cache and page_table must live on one CUDA device")
    shape, torch_dtype = k_cache.shape, k_cache.dtype
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must be [n_pages, page_size, Hkv, D] and alike")
    n_pages, page_size, Hkv, D = shape
    dtype = _KV_DTYPES.get(torch_dtype)
    if dtype is None or v_cache.dtype is not torch_dtype:
        raise TypeError(f"the cache must be bfloat16 or float16, got {torch_dtype} and {v_cache.dtype}")
    kp, kt, kh, kd = k_cache.stride()
    vp, vt, vh, vd = v_cache.stride()
    if kd != 1 or vd != 1:
        raise ValueError("the cache must be contiguous in its last dimension")
    if page_table.dtype is not _I32 or page_table.dim() != 2:
        raise ValueError("page_table must be int32 [B, max_pages]")
    B, max_pages = page_table.shape
    row, entry = page_table.stride()
    if entry != 1 and max_pages > 1:
        raise ValueError("page_table must be contiguous in its last dimension")
    return (k_cache.data_ptr(), v_cache.data_ptr(), dtype, n_pages, page_size, Hkv, D, B, kp, kt, kh, vp, vt, vh,
            page_table.data_ptr(), row if B > 1 else max_pages, max_pages, _int32(ctx_lens, "ctx_lens", index, B)), index


def _tree(tree_parents, index, B):
    if tree_parents is None:
        return 0, 0
    N = tree_parents.shape[-1]
    return _int32(tree_parents, "tree_parents", index, B, N), N


def _raw_stream(index, stream):
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream(stream, index)


def _call(name, index, fn, *args):
    """fn(*args) with CUDA device `index` current; raises on a status."""
    if torch._C._cuda_getDevice() == index:
        st = fn(*args)
    else:
        with torch.cuda.device(index):
            st = fn(*args)
    if st:
        _check(st, name)


def spec_kv_append(k, v, k_cache, v_cache, page_table, ctx_lens, cu_new, q=None, inv_freq=None, interleaved=False,
                   tree_parents=None, positions=None, q_out=None, status_word=None, stream=None):
    """Appends a chunk's keys and values to the paged cache, rotated on the
    way: k and v [T, Hkv, D] packed rows (any token and head strides), cu_new
    [B+1] int32 the rows of each sequence, ctx_lens [B] int32 what the cache
    holds before. With q [T, Hq, D] also rotates the queries, into q_out (or a
    new tensor); q_out may be q. inv_freq: float64 CPU tensor [rotary / 2], the
    angle per position of each rotating pair (rope_inv_freq makes the usual
    one); None leaves keys and queries as they are. tree_parents [B, N]: the
    chunk is a tree, a node's position its context plus its depth. positions
    [T] int32: rotary positions of the caller's own. Returns q_out."""
    if q is None and q_out is not None:
        raise ValueError("q_out is given without q")
    cache, index = _cache_fields(k_cache, v_cache, page_table, ctx_lens)
    Hkv, D, B, dtype = cache[5], cache[6], cache[7], k_cache.dtype
    kp, kt, kh, T, _ = _rows(k, "k", None, Hkv, D, dtype, index)
    vp, vt, vh, _, _ = _rows(v, "v", T, Hkv, D, dtype, index)
    Hq = qp = qt = qh = op = ot = oh = 0
    if q is not None:
        qp, qt, qh, _, Hq = _rows(q, "q", T, None, D, dtype, index)
        if q_out is None:
            q_out = _empty((T, Hq, D), dtype, q.device, stream)
        op, ot, oh, _, _ = _rows(q_out, "q_out", T, Hq, D, dtype, index)
    freq = rotary = 0
    if inv_freq is not None:
        if inv_freq.dtype is not torch.float64 or inv_freq.is_cuda or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            raise ValueError("inv_freq must be a contiguous 1-D float64 CPU tensor")
        freq, rotary = inv_freq.data_ptr(), 2 * inv_freq.numel()
    parents, N = _tree(tree_parents, index, B)
    pos = 0 if positions is None else _int32(positions, "positions", index, T)
    status = _status(status_word, index)
    cu = _int32(cu_new, "cu_new", index, B + 1)
    _call("spec_kv_append", index, (_lib or _load()).spec_kv_append, _pack_append(
        *cache, cu, T, kp, vp, kt, kh, vt, vh, Hq, qp, op, qt, qh, ot, oh, freq, rotary, 1 if interleaved else 0, parents, N,
        pos, status, _raw_stream(index, stream)))
    return q_out


def rope_inv_freq(rotary, base=10000.0):
    """base^(-2i / rotary) for i < rotary / 2, as spec_kv_append takes it."""
    i = torch.arange(rotary // 2, dtype=torch.float64)
    return torch.exp(i * (-2.0 / rotary) * torch.log(torch.tensor(float(base), dtype=torch.float64)))


def spec_paged_attention_workspace_bytes(T, Hq, Hkv, D) -> int:
    return int(_load().spec_paged_attention_workspace_bytes(T, Hq, Hkv, D))


def spec_paged_attention_workspace(T, Hq, Hkv, D, device="cuda"):
    """A workspace for calls of up to T packed rows, its counters zero. Calls
    that may overlap (on different streams) need one each."""
    need = spec_paged_attention_workspace_bytes(T, Hq, Hkv, D)
    if need == 0:
        raise ValueError(f"no workspace for T={T}, Hq={Hq}, Hkv={Hkv}, D={D}")
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    ws[:SV_PAGED_WORKSPACE_HEAD].zero_()
    return ws


def _own_workspace(T, Hq, Hkv, D, device, stream):
    """A workspace of this call alone, on its stream; None where there is none
    (the call itself says why)."""
    if T == 0 or spec_paged_attention_workspace_bytes(T, Hq, Hkv, D) == 0:
        return None
    if stream is None:
        return spec_paged_attention_workspace(T, Hq, Hkv, D, device)
    with torch.cuda.stream(_as_stream(stream, device)):
        return spec_paged_attention_workspace(T, Hq, Hkv, D, device)


def spec_paged_attention(q, k_cache, v_cache, page_table, ctx_lens, cu_new, scale=None, tree_parents=None, out=None,
                         out_lse=None, workspace=None, status_word=None, stream=None, flags=0):
    """Attention of a chunk's tokens (q [T, Hq, D], packed rows of any token
    and head strides) over the paged cache, which holds their keys and values
    already: each token sees its context, itself and the chunk's tokens before
    it, or, with tree_parents [B, N], its ancestors. scale: D ** -0.5 by
    default. out_lse [T, Hq] float32: the rows' log of the sum of exponentials.
    The softmax's weights are rounded to the cache's type before they meet the
    values; scores, sums and the output's sum are fp32.
    workspace: spec_paged_attention_workspace; made anew when None. Returns
    out."""
    cache, index = _cache_fields(k_cache, v_cache, page_table, ctx_lens)
    Hkv, D, B, dtype = cache[5], cache[6], cache[7], k_cache.dtype
    qp, qt, qh, T, Hq = _rows(q, "q", None, None, D, dtype, index)
    if out is None:
        out = _empty((T, Hq, D), dtype, q.device, stream)
    op, ot, oh, _, _ = _rows(out, "out", T, Hq, D, dtype, index)
    lse = 0
    if out_lse is not None:
        if out_lse.dtype is not torch.float32 or out_lse.shape != (T, Hq):
            raise ValueError(f"out_lse must be float32 [{T}, {Hq}]")
        lse = _plain(out_lse, "out_lse", index)
    parents, N = _tree(tree_parents, index, B)
    if workspace is None:
        workspace = _own_workspace(T, Hq, Hkv, D, k_cache.device, stream)
    ws, ws_bytes = (0, 0) if workspace is None else (_plain(workspace, "workspace", index), workspace.numel() * workspace.element_size())
    status = _status(status_word, index)
    cu = _int32(cu_new, "cu_new", index, B + 1)
    scale = D ** -0.5 if scale is None else scale
    _call("spec_paged_attention", index, (_lib or _load()).spec_paged_attention, _pack_attention(
        *cache, cu, T, Hq, qp, op, qt, qh, ot, oh, lse, scale, parents, N, ws, ws_bytes, status, int(flags),
        _raw_stream(index, stream)))
    return out


def spec_kv_commit(k_cache, v_cache, page_table, ctx_lens, n_accepted, tree_parents=None, last_node=None, out_lens=None,
                   status_word=None, stream=None):
    """Keeps what a verify step accepted in the paged cache: the new lengths
    ctx_lens + 1 + n_accepted (into out_lens, which may be ctx_lens, or a new
    tensor), and with tree_parents [B, N] and last_node [B] (as
    spec_verify_tree takes and returns them) the kept path's entries moved
    behind the context. A model's layers share their lengths: each layer's call
    takes those from before the step, so out_lens may be ctx_lens in the last
    one only. Returns out_lens."""
    cache, index = _cache_fields(k_cache, v_cache, page_table, ctx_lens)
    B = cache[7]
    if out_lens is None:
        out_lens = _empty((B,), _I32, ctx_lens.device, stream)
    parents, N = _tree(tree_parents, index, B)
    last = None if last_node is None else _int32(last_node, "last_node", index, B)
    n, lens = _int32(n_accepted, "n_accepted", index, B), _int32(out_lens, "out_lens", index, B)
    status = _status(status_word, index)
    _call("spec_kv_commit", index, (_lib or _load()).spec_kv_commit, _pack_cache(*cache), n, parents, N, last, lens, status,
          _raw_stream(index, stream))
    return out_lens
