"""The calls around sampled decoding beside other work: on other streams, beside
an overlapping verify, from several threads, and in graphs that run together."""
import os
import re
import threading

import pytest
import torch

from speculative_decoding_verification_24_gb300 import (
    spec_kv_pages, spec_lmhead_logits, spec_paged_attention, spec_paged_attention_workspace, spec_sample, spec_truncate_logits,
    spec_verify_ex)
from speculative_decoding_verification_24_gb300.build import CSRC, build

BF16, I32 = torch.bfloat16, torch.int32
DELAY = 50_000_000  # cycles: some 25 ms
NAMES = ("sample", "truncate", "pages", "attention")


@pytest.mark.parametrize("name", ("cut_logits.cu", "kv_pages.cu"))
def test_the_next_kernel_may_start_only_after_the_wait(name):
    with open(os.path.join(CSRC, name)) as f:
        calls = re.findall(r"^\s*(grid_dependency_wait|launch_dependents)\(\);", f.read(), re.M)
    assert calls == ["grid_dependency_wait", "launch_dependents"]


class Calls:
    """Inputs of each call, and its outputs as clones or by name."""

    def __init__(self, seed):
        build()
        assert torch.cuda.is_available(), "GPU tests need a CUDA device"
        dev, g = "cuda", torch.Generator("cuda").manual_seed(seed)
        self.logits = (torch.randn(24, 32001, generator=g, device=dev) * 2).to(BF16)
        self.u = torch.rand(24, generator=g, device=dev)
        self.settings = dict(temperature=torch.linspace(0, 1.5, 24, device=dev), top_p=torch.linspace(0.5, 1, 24, device=dev),
                             top_k=torch.arange(0, 2400, 100, dtype=I32, device=dev))
        B, page, n, Hkv, Hq, D = 16, 16, 5, 2, 8, 64
        ctx = torch.randint(0, 120, (B,), generator=g, device=dev, dtype=I32)
        self.ctx, self.cu = ctx, torch.arange(B + 1, dtype=I32, device=dev) * n
        self.pool = [torch.full((B, 8), -1, dtype=I32, device=dev), torch.zeros(B, dtype=I32, device=dev),
                     torch.randperm(128, generator=g, device=dev).to(I32), torch.tensor([128], dtype=I32, device=dev)]
        self.table = torch.randperm(128, generator=g, device=dev).to(I32).view(B, 8)
        self.k, self.v = (torch.randn(128, page, Hkv, D, generator=g, device=dev).to(BF16) for _ in range(2))
        self.q = torch.randn(B * n, Hq, D, generator=g, device=dev).to(BF16)
        self.slopes = torch.linspace(0.01, 0.5, Hq, device=dev)
        self.ws = spec_paged_attention_workspace(B * n, Hq, Hkv, D)

    def __call__(self, name, stream=None, **outs):
        if name == "sample":
            return spec_sample(self.logits, self.u, **self.settings, stream=stream, **outs)
        if name == "truncate":
            return spec_truncate_logits(self.logits, **self.settings, stream=stream, **outs)
        if name == "attention":
            return spec_paged_attention(self.q, self.k, self.v, self.table, self.ctx, self.cu, stream=stream, workspace=self.ws,
                                        score_cap=10.0, bias_slopes=self.slopes, **outs)
        slots = outs.get("out")
        if slots is None:
            slots = torch.empty(80, dtype=torch.int64, device="cuda")
        # in place, and the same again: the second call finds that each has what it needs
        return spec_kv_pages(*self.pool, self.ctx, self.cu, 16, slots=slots, stream=stream)

    def empty(self, name):
        out = torch.empty_like(self(name))
        return {"out_tokens" if name == "sample" else "out": out}


@pytest.fixture(scope="module")
def calls():
    return Calls(1)


@pytest.mark.gpu
@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ("sample", "truncate", "attention"))
def test_outputs_are_not_memory_that_the_current_stream_still_reads(calls, name, raw):
    side = torch.cuda.Stream()
    want = calls(name).clone()
    size = want.numel() * want.element_size()
    torch.cuda.synchronize()
    for _ in range(3):
        freed = [torch.full((size,), 7, dtype=torch.uint8, device="cuda") for _ in range(2)]
        torch.cuda._sleep(DELAY)
        kept = [t.clone() for t in freed]  # reads them behind the delay
        del freed
        got = calls(name, side.cuda_stream if raw else side)
        side.synchronize()
        torch.cuda.synchronize()
        assert all((t == 7).all() for t in kept)
        assert torch.equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_a_call_between_the_logits_and_an_overlapping_verify(calls, name):
    dev, B, K, d, V = "cuda", 8, 4, 2048, 64000
    g = torch.Generator(dev).manual_seed(5)
    hidden = torch.randn(B * (K + 1), d, generator=g, device=dev).to(BF16)
    W = (torch.randn(d, V, generator=g, device=dev) * d ** -0.5 * 3).to(BF16)
    want_logits = spec_lmhead_logits(hidden, W)
    drafts = want_logits.view(B, K + 1, V).argmax(-1)[:, :K].to(I32).contiguous()
    want = spec_verify_ex(want_logits.view(B, K + 1, V), None, drafts, modes="greedy")
    logits = torch.empty_like(want_logits)
    outs = [(torch.empty_like(want["tokens"]), torch.empty_like(want["n_accepted"])) for _ in range(20)]
    made = calls.empty(name)

    def steps():
        for tokens, n in outs:
            logits.zero_()  # stale logits accept nothing
            spec_lmhead_logits(hidden, W, out=logits)
            calls(name, **made)
            spec_verify_ex(logits.view(B, K + 1, V), None, drafts, modes="greedy", overlap_previous=True, out_tokens=tokens,
                           out_n_accepted=n)

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


@pytest.mark.gpu
def test_logits_that_the_call_before_writes_and_a_cut_that_the_next_one_reads():
    """LM head, cut in place, draw and verify in a row, without waits of the host."""
    build()
    dev, B, K, d, V = "cuda", 6, 3, 256, 20000
    g = torch.Generator(dev).manual_seed(6)
    W = (torch.randn(d, V, generator=g, device=dev) * d ** -0.5 * 3).to(BF16)
    u = torch.rand(B, K + 1, generator=g, device=dev)
    for _ in range(20):
        hidden = torch.randn(B * (K + 1), d, generator=g, device=dev).to(BF16)
        logits = spec_lmhead_logits(hidden, W).view(B, K + 1, V)
        whole = logits.clone()
        spec_truncate_logits(logits, top_k=1, out=logits)
        tokens = spec_sample(logits, u)
        n = spec_verify_ex(logits, None, tokens[:, :K].contiguous(), modes="greedy")["n_accepted"]
        first = whole.float().argmax(-1).to(I32)
        assert torch.equal(tokens, first) and (n == K).all()


@pytest.mark.gpu
def test_threads_with_streams_of_their_own():
    made = [Calls(20 + i) for i in range(4)]
    want = [{n: c(n).clone() for n in NAMES} for c in made]
    torch.cuda.synchronize()
    bad = []

    def work(c, ref):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                outs = [(n, c(n)) for _ in range(25) for n in NAMES]
            stream.synchronize()
            bad.extend(n for n, out in outs if not torch.equal(out, ref[n]))
        except Exception as e:  # noqa: BLE001
            bad.append(e)

    threads = [threading.Thread(target=work, args=x) for x in zip(made, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert bad == []


@pytest.mark.gpu
def test_graphs_that_run_together():
    made = [Calls(30 + i) for i in range(2)]
    want = [{n: c(n).clone() for n in NAMES} for c in made]
    outs = [{n: c.empty(n) for n in NAMES} for c in made]
    torch.cuda.synchronize()
    graphs, streams = [], [torch.cuda.Stream() for _ in made]
    for c, o in zip(made, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            for _ in range(5):
                for n in NAMES:
                    c(n, **o[n])
    for _ in range(10):
        for o in outs:
            for n in NAMES:
                for t in o[n].values():
                    t.zero_()
        torch.cuda.synchronize()
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            for n in NAMES:
                assert all(torch.equal(t, w[n]) for t in o[n].values())
