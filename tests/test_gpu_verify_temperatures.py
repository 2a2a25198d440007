"""A batch of sequences with a temperature of their own each is verified as a call
per sequence verifies it."""
import math

import pytest
import torch

from speculative_decoding_verification_24_gb300 import binding, spec_sample, spec_truncate_logits, spec_verify, spec_verify_ex, spec_verify_plan
from speculative_decoding_verification_24_gb300.build import LIB_DEBUG, build

pytestmark = pytest.mark.gpu

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
BAD_MODE, BAD_SETTING = 16, 1024


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def batch(B, K, V, dtype, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    target = torch.randn(B, K + 1, V, generator=g, device="cuda") * 2
    draft = target[:, :K] + 0.5 * torch.randn(B, K, V, generator=g, device="cuda")
    drafts = (draft + 0.5 * torch.randn(B, K, V, generator=g, device="cuda")).argmax(-1).to(I32)
    return target.to(dtype), draft.to(dtype), drafts


NAMES = ("tokens", "n_accepted", "p_target", "p_draft", "residual_mass", "draw_edges")


def one_by_one(target, draft, drafts, T, modes=None, draft_lens=None, **kw):
    """A call per sequence with its temperature as a number; at 0 a greedy one."""
    rows = []
    for b, t in enumerate(T.tolist()):
        mode = "greedy" if t == 0 or (modes is not None and modes[b] == 0) else "sample"
        rows.append(spec_verify_ex(target[b:b + 1], draft[b:b + 1], drafts[b:b + 1], t or 1.0, mode, debug=True,
                                   seq_ids=torch.tensor([b], dtype=torch.int64, device="cuda").view(torch.uint64),
                                   draft_lens=None if draft_lens is None else draft_lens[b:b + 1].contiguous(), **kw))
    out = {n: torch.cat([r[n] for r in rows]) for n in NAMES}
    out["flags"] = 0
    for r in rows:
        out["flags"] |= r["status_word"].item()
    return out


def same(got, want):
    """To the bit: clusters of one size split a row alike. Flags too: a distribution of
    one token may leave no residual to draw from, which a flag says."""
    if "flags" in want:
        assert got["status_word"].item() == want["flags"]
    for n in NAMES:
        assert torch.equal(got[n].nan_to_num(nan=-7.0), want[n].nan_to_num(nan=-7.0)), n


T8 = (1.0, 0.5, 0.0, 1.7, 0.8, 2.0 ** -20, 100.0, 0.9)


@pytest.mark.parametrize("overlap", (False, True))
@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "fp32"))
@pytest.mark.parametrize("K,V,cs", ((1, 2, 1), (4, 1001, 1), (5, 32000, 4), (8, 50003, 8)))
def test_as_a_call_per_sequence(K, V, cs, dtype, overlap):
    target, draft, drafts = batch(8, K, V, dtype, K)
    T = torch.tensor(T8, device="cuda")
    got = spec_verify_ex(target, draft, drafts, T, seed=5, cluster_size=cs, debug=True, overlap_previous=overlap)
    torch.cuda.synchronize()
    same(got, one_by_one(target, draft, drafts, T, seed=5, cluster_size=cs))


def test_beside_modes_and_draft_counts():
    target, draft, drafts = batch(8, 5, 9000, BF16, 3)
    T = torch.tensor(T8, device="cuda")
    modes = torch.tensor([1, 0, 1, 1, 0, 1, 1, 0], dtype=I32, device="cuda")
    lens = torch.tensor([5, 3, 2, 0, 5, 1, 4, 0], dtype=I32, device="cuda")
    T[1] = math.nan  # (a greedy sequence's is not looked at)
    got = spec_verify_ex(target, draft, drafts, T, modes, seed=6, cluster_size=2, debug=True, draft_lens=lens)
    T[1] = 1.0
    same(got, one_by_one(target, draft, drafts, T, modes.tolist(), lens, seed=6, cluster_size=2))
    # a greedy call looks at none
    got = spec_verify(target, None, drafts, torch.full((8,), math.nan, device="cuda"), "greedy")
    want = spec_verify(target, None, drafts, 1.0, "greedy")
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("B", (1, 19, 64, 300))
def test_sizes_that_choose_their_clusters(B):
    """No sequences per cluster, however large the batch; tokens as with one
    temperature where all are the same."""
    target, draft, drafts = batch(B, 3, 4001, F32, B)
    T = torch.full((B,), 0.75, device="cuda")
    assert not spec_verify_plan(target, draft, drafts, T)["grouped"]
    tokens, n = spec_verify(target, draft, drafts, T, seed=9)
    want = spec_verify_ex(target, draft, drafts, 0.75, seed=9, seqs_per_cluster=1)
    assert torch.equal(tokens, want["tokens"]) and torch.equal(n, want["n_accepted"])


def test_temperatures_out_of_range():
    target, draft, drafts = batch(8, 3, 700, F32, 1)
    bad = torch.tensor([1.0, -1.0, math.nan, math.inf, -math.inf, 1e-39, 0.5, 3e38], device="cuda")
    got = spec_verify_ex(target, draft, drafts, bad, cluster_size=1, debug=True)
    assert got["status_word"].item() == BAD_SETTING
    ok = [0, 6, 7]
    assert [b for b, n in enumerate(got["n_accepted"].tolist()) if n >= 0] == ok
    for b in set(range(8)) - set(ok):
        assert (got["tokens"][b] == -1).all() and got["p_target"][b].isnan().all() and got["draw_edges"][b].isnan().all()
    fine = torch.where(torch.isin(torch.arange(8, device="cuda"), torch.tensor(ok, device="cuda")), bad, 1.0)
    want = one_by_one(target, draft, drafts, fine, cluster_size=1)
    same({n: got[n][ok] for n in NAMES}, {n: want[n][ok] for n in NAMES})


def test_refusals():
    target, draft, drafts = batch(4, 3, 700, F32, 1)
    T = torch.ones(4, device="cuda")
    with pytest.raises(binding.SpecVerifyError) as e:
        spec_verify_ex(target, draft, drafts, T, seqs_per_cluster=2)
    assert e.value.status == 10
    for bad, error in ((T.double(), TypeError), (T[:3], ValueError), (T.cpu(), ValueError), (torch.ones(8, device="cuda")[::2], ValueError)):
        with pytest.raises(error):
            spec_verify_ex(target, draft, drafts, bad)
        with pytest.raises(error):
            spec_verify(target, draft, drafts, bad)


def test_debug_build_reads_nothing_else():
    target, draft, drafts = batch(8, 4, 5000, BF16, 2)
    T = torch.tensor(T8, device="cuda")
    lib = binding.load_library(LIB_DEBUG)
    got = spec_verify_ex(target, draft, drafts, T, seed=3, cluster_size=2, debug=True, lib=lib)
    want = spec_verify_ex(target, draft, drafts, T, seed=3, cluster_size=2, debug=True)
    same(got, dict(want, flags=want["status_word"].item()))


def test_graph_takes_new_temperatures():
    target, draft, drafts = batch(8, 4, 5000, BF16, 2)
    T = torch.ones(8, device="cuda")
    out = torch.empty(8, 5, dtype=I32, device="cuda"), torch.empty(8, dtype=I32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        spec_verify(target, draft, drafts, T, seed=3, out_tokens=out[0], out_n_accepted=out[1])
    for scale in (1.0, 0.3):
        T.copy_(torch.tensor(T8, device="cuda") * scale)
        graph.replay()
        want = spec_verify(target, draft, drafts, T, seed=3)
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "fp32"))
def test_drafts_cut_and_verified_by_their_own_temperatures(dtype):
    """From the draw to the verify step with one tensor of temperatures, one of them
    0: a sequence's text is that of a call of its own, and lies in its cut."""
    B, K, V = 24, 4, 8000
    target, draft, _ = batch(B, K, V, dtype, 4)
    g = torch.Generator().manual_seed(5)
    u = torch.rand(B, K, generator=g).cuda()
    T = torch.tensor([0.0, 0.6, 0.8, 1.0, 1.3, 2.5])[torch.arange(B) % 6].cuda()
    p = torch.tensor([0.9, 1.0, 0.7, 0.95])[torch.arange(B) % 4].cuda()
    settings = dict(temperature=T, top_k=60, top_p=p)
    lp = torch.empty(B, K, device="cuda")
    drafts = spec_sample(draft, u, **settings, out_logprobs=lp)
    cut_d, cut_t = spec_truncate_logits(draft, **settings), spec_truncate_logits(target, **settings)
    got = spec_verify_ex(cut_t, cut_d, drafts, T, seed=7, debug=True, cluster_size=2)
    same(got, one_by_one(cut_t, cut_d, drafts, T, seed=7, cluster_size=2))
    tokens, n = got["tokens"].tolist(), got["n_accepted"].tolist()
    assert max(n) > 0
    for b in range(B):
        for i in range(n[b] + 1):
            assert cut_t[b, i, tokens[b][i]].item() > -math.inf
    # the verify step's probabilities of the drafts are those that they were drawn by
    # (2^-20: its own are right to 1e-6 here, the logarithm is fp32)
    drawn = (T > 0)[:, None].expand(B, K)
    assert ((got["p_draft"].log() - lp).abs() <= 2.0 ** -20 * (1 + lp.abs()))[drawn].all()


def test_the_example_takes_settings_by_sequence():
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import paged_decode as ex
    B, L_max, kw = 6, 200, dict(score_cap=30.0, biased=True, pooled=True)
    model, drafter = ex.Decoder(B, L_max, **kw), ex.Decoder(B, L_max, layers=1, **kw)
    prompts = ex.example_prompts(B, model.V)
    text, lens = ex.start(model, prompts, L_max)
    ex.start(drafter, prompts, L_max)
    g = torch.Generator(device="cuda").manual_seed(5)
    T = torch.tensor([0.0, 0.5, 0.8, 1.0, 1.4, 0.0], device="cuda")
    k = torch.tensor([0, 20, 40, 60, 10, 5], dtype=I32, device="cuda")
    for i in range(10):
        before = lens.clone()
        n, rows = ex.step_sample(model, drafter, text, lens, torch.rand(4, B, device="cuda", generator=g), i, temperature=T, top_k=k)
        assert (n >= 0).all() and torch.equal(lens, before + n + 1)
        kept = (rows > float("-inf")).sum(-1)
        assert (kept[T == 0] == 1).all() and (kept[k > 0] <= k[k > 0][:, None]).all()
        for b in range(B):
            for j in range(int(n[b]) + 1):
                assert rows[b, j, text[b, before[b] + j]] > float("-inf")
