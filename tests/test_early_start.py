"""Calls that start beside the work ahead of them. A kernel that waits for all of
the work before it may let the next one start only after that wait: a verify
call with SV_ARG_OVERLAP_PREVIOUS reads its inputs without waiting, and the
work before the call in between may have written them."""
import os
import re

import pytest
import torch

from speculative_decoding_verification_24_gb300 import (
    rope_inv_freq, spec_commit, spec_kv_append, spec_kv_commit, spec_lmhead_logits, spec_paged_attention,
    spec_paged_attention_workspace, spec_prompt_lookup, spec_verify_ex)
from speculative_decoding_verification_24_gb300.build import CSRC, build

WAITING = {"kv_cache.cu": 2, "paged_attention.cu": 1, "prompt_lookup.cu": 2}  # kernels that wait for all of their work


@pytest.mark.parametrize("name", WAITING)
def test_the_next_kernel_may_start_only_after_the_wait(name):
    with open(os.path.join(CSRC, name)) as f:
        calls = re.findall(r"^\s*(grid_dependency_wait|launch_dependents)\(\);", f.read(), re.M)
    assert calls == ["grid_dependency_wait", "launch_dependents"] * WAITING[name]


@pytest.fixture(scope="module")
def between():
    """Calls that neither read nor write what the LM head and the verify call do."""
    build()
    dev, B, K, page, Hkv, D, Hq = "cuda", 8, 4, 16, 2, 64, 8
    g = torch.Generator(dev).manual_seed(3)
    kc, vc = (torch.randn(64, page, Hkv, D, generator=g, device=dev).to(torch.bfloat16) for _ in range(2))
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    table = torch.arange(64, dtype=torch.int32, device=dev).view(B, 8)
    ctx, cu = ints(*range(10, 90, 10)), torch.arange(B + 1, dtype=torch.int32, device=dev) * 5
    qkv = torch.randn(5 * B, Hq + 2 * Hkv, D, generator=g, device=dev).to(torch.bfloat16)
    q, k, v = qkv[:, :Hq].contiguous(), qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    ws, q_out, out = spec_paged_attention_workspace(5 * B, Hq, Hkv, D), torch.empty_like(q), torch.empty_like(q)
    text, lens = torch.randint(0, 9, (B, 256), generator=g, device=dev, dtype=torch.int32), ints(*[100] * B)
    tokens, zeros, lens_out = torch.zeros(B, K + 1, dtype=torch.int32, device=dev), ints(*[0] * B), ints(*[0] * B)
    drafts = torch.empty(B, K, dtype=torch.int32, device=dev), torch.empty(B, dtype=torch.int32, device=dev)
    freq = rope_inv_freq(D)
    return {
        "append": lambda: spec_kv_append(k, v, kc, vc, table, ctx, cu, q=q, q_out=q_out, inv_freq=freq),
        "attention": lambda: spec_paged_attention(q, kc, vc, table, ctx, cu, out=out, workspace=ws),
        "keep": lambda: spec_kv_commit(kc, vc, table, ctx, zeros, out_lens=lens_out),
        "lookup": lambda: spec_prompt_lookup(text, lens, n_drafts=K, out_drafts=drafts[0], out_n_drafts=drafts[1]),
        "commit": lambda: spec_commit(text, lens, tokens, zeros, out_n_committed=lens_out),
    }


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["append", "attention", "keep", "lookup", "commit"])
def test_a_call_between_the_logits_and_an_overlapping_verify(between, name):
    dev, B, K, d, V = "cuda", 8, 4, 2048, 64000
    g = torch.Generator(dev).manual_seed(5)
    hidden = torch.randn(B * (K + 1), d, generator=g, device=dev).to(torch.bfloat16)
    W = (torch.randn(d, V, generator=g, device=dev) * d ** -0.5 * 3).to(torch.bfloat16)
    want_logits = spec_lmhead_logits(hidden, W)
    # the target's own tokens, so that every row is read and decides
    drafts = want_logits.view(B, K + 1, V).argmax(-1)[:, :K].to(torch.int32).contiguous()
    want = spec_verify_ex(want_logits.view(B, K + 1, V), None, drafts, modes="greedy")
    logits = torch.empty_like(want_logits)
    outs = [(torch.empty_like(want["tokens"]), torch.empty_like(want["n_accepted"])) for _ in range(20)]

    def steps():
        for tokens, n in outs:
            logits.zero_()  # stale logits accept nothing
            spec_lmhead_logits(hidden, W, out=logits)
            between[name]()
            spec_verify_ex(logits.view(B, K + 1, V), None, drafts, modes="greedy", overlap_previous=True, out_tokens=tokens,
                           out_n_accepted=n)

    between[name]()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps()
    for run in (steps, graph.replay):
        for tokens, n in outs:
            tokens.fill_(-7), n.fill_(-7)
        run()
        torch.cuda.synchronize()
        assert int(want["n_accepted"].min()) == K
        for tokens, n in outs:
            assert torch.equal(tokens, want["tokens"]) and torch.equal(n, want["n_accepted"])
