"""The example decoder that samples: pages from a pool, capped scores and a bias
by distance, drafts drawn from a smaller model's cut rows, both models' rows cut
and verified."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

from speculative_decoding_verification_24_gb300.build import build

pytestmark = pytest.mark.gpu

B, L_MAX, KW = 8, 256, dict(score_cap=30.0, biased=True, pooled=True)


@pytest.fixture(scope="module")
def ex():
    build()
    import paged_decode
    return paged_decode


def check_pool(model):
    table, held, free, n_free = model.pool
    owned = [table[b, :held[b]].tolist() for b in range(model.B)]
    assert sorted(sum(owned, []) + free[:n_free.item()].tolist()) == list(range(free.numel()))
    return held


def test_one_token_kept_is_greedy_decoding(ex):
    """Rows cut to their first token accept a draft exactly where it is the
    target's: the text is that of decoding a token at a time."""
    plain = ex.Decoder(B, L_MAX, **KW)
    prompts = ex.example_prompts(B, plain.V)
    want, want_lens = ex.start(plain, prompts, L_MAX)
    gaps = []
    for _ in range(60):
        _, logits = ex.step_plain(plain, want, want_lens)
        top = logits.topk(2, dim=1).values
        gaps.append((top[:, 0] - top[:, 1]) / logits.abs().amax(1))
    check_pool(plain)
    model, drafter = ex.Decoder(B, L_MAX, **KW), ex.Decoder(B, L_MAX, **KW)  # the same weights: drafts are right
    text, lens = ex.start(model, prompts, L_MAX)
    ex.start(drafter, prompts, L_MAX)
    accepted = 0
    u = torch.rand(4, B, device="cuda")
    for i in range(20):
        n, _ = ex.step_sample(model, drafter, text, lens, u, i, temperature=1.0, top_k=1)
        assert torch.equal(model.ctx, lens - 1) and torch.equal(drafter.ctx, lens - 1)
        accepted += int(n.clamp(min=0).sum())
    assert accepted > 20 * B  # of 80 per sequence
    check_pool(model)
    check_pool(drafter)
    text, lens, want, want_lens, gaps = text.cpu(), lens.cpu(), want.cpu(), want_lens.cpu(), torch.stack(gaps).cpu()
    whole = 0
    for b, p in enumerate(prompts):
        n = min(int(lens[b]), int(want_lens[b]))
        differ = (text[b, :n] != want[b, :n]).nonzero()
        whole += len(differ) == 0
        if len(differ):  # only where two tokens are as good as equal: bf16 activations (2^-8) batched in another way
            assert float(gaps[int(differ[0]) - len(p), b]) < 2.0 ** -6, (b, int(differ[0]))
    assert whole >= B // 2


def test_sampled_text_stays_within_the_cut(ex):
    model, drafter = ex.Decoder(B, L_MAX, **KW), ex.Decoder(B, L_MAX, layers=1, **KW)
    prompts = ex.example_prompts(B, model.V)
    text, lens = ex.start(model, prompts, L_MAX)
    ex.start(drafter, prompts, L_MAX)
    g = torch.Generator(device="cuda").manual_seed(5)
    for i in range(25):
        u = torch.rand(4, B, device="cuda", generator=g)
        before = lens.clone()
        n, rows = ex.step_sample(model, drafter, text, lens, u, i, temperature=0.8, top_k=40, top_p=0.9)
        assert (n >= 0).all() and torch.equal(lens, before + n + 1)
        kept = (rows > float("-inf")).sum(-1)
        assert (kept >= 1).all() and (kept <= 40).all()
        for b in range(B):
            for j in range(int(n[b]) + 1):
                assert rows[b, j, text[b, before[b] + j]] > float("-inf")
        held = check_pool(model)
        assert (held * model.page >= model.ctx).all()
