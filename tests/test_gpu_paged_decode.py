"""The example decoder end to end: drafting, appending, attention over the
paged cache, verification and commit give the text that decoding a token at a
time gives, for chains and for trees of drafts."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

from speculative_decoding_verification_24_gb300.build import build

pytestmark = pytest.mark.gpu

B, L_MAX, TOKENS = 8, 512, 120


@pytest.fixture(scope="module")
def plain():
    build()
    import paged_decode as ex
    model = ex.Decoder(B, L_MAX)
    prompts = ex.example_prompts(B, model.V)
    text, lens = ex.start(model, prompts, L_MAX)
    gaps = []  # how far the chosen token's logit lies above the next one's
    for _ in range(TOKENS):
        _, logits = ex.step_plain(model, text, lens)
        top = logits.topk(2, dim=1).values
        gaps.append((top[:, 0] - top[:, 1]) / logits.abs().amax(1))
    torch.cuda.synchronize()
    return prompts, text.cpu(), lens.cpu(), torch.stack(gaps).cpu()


@pytest.mark.parametrize("mode", ["chain", "tree"])
def test_drafted_decoding_equals_plain_decoding(plain, mode):
    import paged_decode as ex
    prompts, want, want_lens, gaps = plain
    model = ex.Decoder(B, L_MAX)
    text, lens = ex.start(model, prompts, L_MAX)
    accepted = 0
    for _ in range(TOKENS // 2):
        n, _ = ex.STEPS[mode](model, text, lens)
        assert torch.equal(model.ctx, lens - 1)  # cache and text stay in step
        accepted += int(n.clamp(min=0).sum())
    text, lens = text.cpu(), lens.cpu()
    assert accepted > 0  # drafts were kept, so the moved entries were read
    whole = 0
    for b, p in enumerate(prompts):
        n = min(int(lens[b]), int(want_lens[b]))
        differ = (text[b, :n] != want[b, :n]).nonzero()
        whole += len(differ) == 0
        if len(differ):
            # only where two tokens are as good as equal: activations are
            # rounded to bf16 (2^-8) in either way of batching
            assert float(gaps[int(differ[0]) - len(p), b]) < 2.0 ** -6, (b, int(differ[0]))
    assert whole >= B // 2


@pytest.mark.parametrize("mode", ["chain", "tree"])
def test_drafted_decoding_up_to_the_end_of_the_text(mode):
    # the drafts of the last steps lie past the text's last place, and a full
    # text's steps change nothing
    import paged_decode as ex
    build()
    L, steps = 128, 124  # whole pages
    texts, gaps = {}, []
    for way in ("plain", mode):
        model = ex.Decoder(B, L)
        prompts = ex.example_prompts(B, model.V)
        text, lens = ex.start(model, prompts, L)
        for _ in range(steps):
            full = (lens == L).tolist()
            before = text[lens == L]
            _, logits = ex.STEPS[way](model, text, lens)
            assert torch.equal(text[torch.tensor(full, device="cuda")], before)
            assert torch.equal(model.ctx, lens - 1)
            if way == "plain":
                top = logits.topk(2, dim=1).values
                gaps.append((top[:, 0] - top[:, 1]) / logits.abs().amax(1))
        assert (lens == L).all()
        texts[way] = text.cpu()
    gaps, whole = torch.stack(gaps).cpu(), 0
    for b, p in enumerate(prompts):
        differ = (texts["plain"][b] != texts[mode][b]).nonzero()
        whole += len(differ) == 0
        if len(differ):  # only where two tokens are as good as equal, as above
            assert float(gaps[int(differ[0]) - len(p), b]) < 2.0 ** -6, (b, int(differ[0]))
    assert whole >= B // 2
