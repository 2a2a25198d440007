"""Calls on another stream than the current one: the outputs they make are not
memory that the current stream's work still uses."""
import pytest
import torch

from speculative_decoding_verification_24_gb300 import (
    rope_inv_freq, spec_commit, spec_kv_append, spec_kv_commit, spec_lmhead_logits, spec_paged_attention, spec_prompt_lookup,
    spec_verify, spec_verify_ex, spec_verify_lmhead, spec_verify_tree)
from speculative_decoding_verification_24_gb300.build import build

pytestmark = pytest.mark.gpu

BF16, I32 = torch.bfloat16, torch.int32
DELAY = 50_000_000  # cycles: some 25 ms


@pytest.fixture(scope="module")
def calls():
    """name -> a call that makes its outputs, on the stream given, and returns them."""
    build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    dev, B, K, V, d, page, Hkv, Hq, D = "cuda", 16, 4, 4096, 256, 16, 2, 8, 64
    g = torch.Generator(dev).manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    logits, draft = rnd(B, K + 1, V), rnd(B, K, V)
    x = torch.randint(0, V, (B, K), generator=g, device=dev, dtype=I32)
    hidden, W = rnd(B, K + 1, d).to(BF16), (rnd(d, V) * d ** -0.5).to(BF16)
    nodes = torch.randint(0, V, (B, K + 1), generator=g, device=dev, dtype=I32)
    parents = torch.tensor([-1, 0, 0, 1, 2], dtype=I32, device=dev).expand(B, -1).contiguous()
    text, lens = torch.randint(0, 9, (B, 256), generator=g, device=dev, dtype=I32), torch.full((B,), 100, dtype=I32, device=dev)
    zeros, ctx = torch.zeros(B, dtype=I32, device=dev), torch.full((B,), 20, dtype=I32, device=dev)
    kc, vc = rnd(2 * B, page, Hkv, D).to(BF16), rnd(2 * B, page, Hkv, D).to(BF16)
    table, cu = torch.arange(2 * B, dtype=I32, device=dev).view(B, 2), torch.arange(B + 1, dtype=I32, device=dev)
    q, k, v = rnd(B, Hq, D).to(BF16), rnd(B, Hkv, D).to(BF16), rnd(B, Hkv, D).to(BF16)
    freq = rope_inv_freq(D)
    tokens = torch.zeros(B, K + 1, dtype=I32, device=dev)
    return {
        "verify": lambda s: spec_verify(logits, draft, x, stream=s),
        "verify_ex": lambda s: tuple(t for t in spec_verify_ex(logits, draft, x, debug=True, stream=s).values()),
        "tree": lambda s: spec_verify_tree(logits, nodes, parents, stream=s),
        "lookup": lambda s: spec_prompt_lookup(text, lens, stream=s),
        "commit": lambda s: (spec_commit(text, lens, tokens, zeros, stream=s),),
        "logits": lambda s: (spec_lmhead_logits(hidden, W, stream=s),),
        "lmhead": lambda s: spec_verify_lmhead(hidden, W, draft, x, stream=s),
        "append": lambda s: (spec_kv_append(k, v, kc, vc, table, ctx, cu, q=q, inv_freq=freq, stream=s),),
        "attention": lambda s: (spec_paged_attention(q, kc, vc, table, ctx, cu, stream=s),),
        "keep": lambda s: (spec_kv_commit(kc, vc, table, ctx, zeros, stream=s),),
    }


NAMES = ("verify", "verify_ex", "tree", "lookup", "commit", "logits", "lmhead", "append", "attention", "keep")


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_outputs_are_not_memory_that_the_current_stream_still_reads(calls, name, raw):
    side = torch.cuda.Stream()
    want = [t.clone() for t in calls[name](None)]
    sizes = [t.numel() * t.element_size() for t in want]
    torch.cuda.synchronize()
    for _ in range(3):
        freed = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes * 2]
        torch.cuda._sleep(DELAY)
        kept = [t.clone() for t in freed]  # reads them behind the delay
        del freed
        got = calls[name](side.cuda_stream if raw else side)
        side.synchronize()
        torch.cuda.synchronize()
        assert all((t == 7).all() for t in kept)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_outputs_that_were_dropped_are_not_handed_out_while_the_call_writes_them(calls, name):
    side = torch.cuda.Stream()
    sizes = [t.numel() * t.element_size() for t in calls[name](None)]
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(DELAY)
        calls[name](side)
        fresh = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes * 2]
        side.synchronize()
        torch.cuda.synchronize()
        assert all((t == 7).all() for t in fresh)


def test_threads_with_streams_and_workspaces_of_their_own():
    import threading
    from test_gpu_paged_attention import Case
    from speculative_decoding_verification_24_gb300 import spec_paged_attention_workspace
    build()
    cases = [Case([(700, 5), (0, 200), (3000, 1)], seed=50 + i) for i in range(4)]
    want = [c.run() for c in cases]
    torch.cuda.synchronize()
    bad = []

    def work(c, ref):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                ws = spec_paged_attention_workspace(c.q.shape[0], 8, 2, 128)
                outs = [spec_paged_attention(c.q, c.k, c.v, *c.args, workspace=ws) for _ in range(50)]
            stream.synchronize()
            bad.extend(i for i, out in enumerate(outs) if not torch.equal(out, ref))
        except Exception as e:  # noqa: BLE001
            bad.append(e)

    threads = [threading.Thread(target=work, args=x) for x in zip(cases, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert bad == []


@pytest.mark.parametrize("raw", [0, 1])
def test_the_default_streams_handle(raw):
    from test_gpu_paged_attention import Case
    from speculative_decoding_verification_24_gb300 import binding
    build()
    assert binding._as_stream(raw, "cuda:0") == torch.cuda.default_stream()
    c = Case([(3000, 5), (100, 70)], seed=51)
    want = c.run()
    size = binding.spec_paged_attention_workspace_bytes(c.q.shape[0], 8, 2, 128)
    for _ in range(5):
        junk = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda._sleep(DELAY // 10)
        del junk  # the call's own workspace is this memory, its counters zeroed on the same stream
        assert torch.equal(c.run(stream=raw), want)
