"""Greedy speculative decoding with a paged key/value cache, all on the GPU.

    python examples/paged_decode.py [--mode plain|chain|tree|sample] [--steps N]

A small decoder with random weights runs over a cache of pages handed out in
no order. A step drafts from each sequence's own text (spec_prompt_lookup),
appends the last token and the drafts to the cache with the rotation applied
(spec_kv_append), attends from them over the cache (spec_paged_attention),
verifies with the LM head (spec_verify_lmhead; or spec_lmhead_logits and
spec_verify_tree), and keeps what was accepted in the text (spec_commit) and in
the cache (spec_kv_commit). "plain" decodes a token at a time with the same
calls; both give the same text, the drafted ways in fewer steps.

"sample" draws: a smaller model drafts from its rows cut by temperature, top-k and
top-p (spec_sample), the rows of both are cut alike (spec_truncate_logits) and
verified by the sampling rule (spec_verify). There the scores are capped, keys are
biased by distance instead of rotated, and the pages come from a pool that
spec_kv_pages hands out.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from speculative_decoding_verification_24_gb300 import (  # noqa: E402
    rope_inv_freq, spec_commit, spec_kv_append, spec_kv_commit, spec_kv_pages, spec_lmhead_logits, spec_paged_attention,
    spec_paged_attention_workspace, spec_prompt_lookup, spec_sample, spec_truncate_logits, spec_verify, spec_verify_lmhead,
    spec_verify_lmhead_workspace_bytes, spec_verify_tree)

BF16 = torch.bfloat16
CHUNK = 32  # tokens of a step's chunk at most


class Decoder:
    """A decoder of pre-norm layers whose keys and values live in a paged
    cache of its own."""

    def __init__(self, B, L_max, layers=2, d=512, Hq=8, Hkv=2, D=64, V=1024, page=16, seed=0, device="cuda", score_cap=None,
                 biased=False, pooled=False):
        g = torch.Generator(device=device).manual_seed(seed)
        w = lambda *s: (torch.randn(*s, generator=g, device=device) * s[-2] ** -0.5).to(BF16)  # noqa: E731
        self.B, self.d, self.V, self.heads, self.device = B, d, V, (Hq, Hkv, D), device
        self.embed = torch.randn(V, d, generator=g, device=device).to(BF16)
        self.head = w(d, V) * 4
        self.layers = [dict(qkv=w(d, (Hq + 2 * Hkv) * D), out=w(Hq * D, d), up=w(d, 4 * d), down=w(4 * d, d))
                       for _ in range(layers)]
        # the last steps' drafts lie past the text's last place; a chunk without
        # room for all of its tokens would be left out as a whole
        per_seq = -(-(L_max + CHUNK) // page)
        self.caches = [tuple(torch.empty(B * per_seq, page, Hkv, D, dtype=BF16, device=device) for _ in range(2))
                       for _ in range(layers)]
        self.table = torch.randperm(B * per_seq, generator=g, device=device).to(torch.int32).view(B, per_seq)
        self.ctx = torch.zeros(B, dtype=torch.int32, device=device)  # tokens in the cache
        self.pool = None
        if pooled:  # the same pages, none of them anyone's yet
            self.pool = [torch.full_like(self.table, -1), torch.zeros_like(self.ctx), self.table.flatten(),
                         torch.full((1,), B * per_seq, dtype=torch.int32, device=device)]
            self.table, self.page = self.pool[0], page
        self.score_cap = score_cap
        self.slopes = torch.tensor([2.0 ** (-8 * (h + 1) / Hq) for h in range(Hq)], device=device) if biased else None
        self.inv_freq = None if biased else rope_inv_freq(D)
        self.workspace = spec_paged_attention_workspace(B * L_max, Hq, Hkv, D, device=device)

    @staticmethod
    def norm(x):
        x = x.float()
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(BF16)

    def forward(self, tokens, cu, parents=None):
        """Final hidden states [T, d] of the packed new tokens, whose keys and
        values go into the cache behind self.ctx."""
        Hq, Hkv, D = self.heads
        if self.pool is not None:
            spec_kv_pages(*self.pool, self.ctx, cu, self.page)
        x = self.embed[tokens.long()]
        for layer, (kc, vc) in zip(self.layers, self.caches):
            qkv = (self.norm(x) @ layer["qkv"]).view(-1, Hq + 2 * Hkv, D)
            q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
            q = spec_kv_append(k, v, kc, vc, self.table, self.ctx, cu, q=q, inv_freq=self.inv_freq, tree_parents=parents)
            a = spec_paged_attention(q, kc, vc, self.table, self.ctx, cu, tree_parents=parents, workspace=self.workspace,
                                     score_cap=self.score_cap, bias_slopes=self.slopes)
            x = x + a.view(-1, Hq * D) @ layer["out"]
            x = x + torch.nn.functional.gelu(self.norm(x) @ layer["up"]) @ layer["down"]
        return self.norm(x)

    def keep(self, n_accepted, parents=None, last_node=None):
        """The cache after a verify step: a chain's entries lie where they
        belong, a tree's move in every layer."""
        lens = torch.empty_like(self.ctx)
        for kc, vc in self.caches[:1] if parents is None else self.caches:
            spec_kv_commit(kc, vc, self.table, self.ctx, n_accepted, tree_parents=parents, last_node=last_node, out_lens=lens)
        self.ctx = lens

    def commit(self, text, lens, tokens, n_accepted, parents=None, last_node=None):
        """What was accepted, in the cache and in the text. A text that is full
        takes no more, and the cache stays with it."""
        self.keep(n_accepted, parents, last_node)
        spec_commit(text, lens, tokens, n_accepted)
        torch.minimum(self.ctx, lens - 1, out=self.ctx)


def start(model, prompts, L_max):
    """Texts and lengths on the GPU, and the cache filled with all but each
    prompt's last token."""
    dev = model.device
    text = torch.zeros(model.B, L_max, dtype=torch.int32, device=dev)
    for b, p in enumerate(prompts):
        text[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    lens = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device=dev)
    packed = torch.tensor([t for p in prompts for t in p[:-1]], dtype=torch.int32, device=dev)
    cu = torch.cat([torch.zeros(1, dtype=torch.int32, device=dev), (lens - 1).cumsum(0).to(torch.int32)])
    model.forward(packed, cu)
    model.ctx = lens - 1
    return text, lens


def last_tokens(text, lens):
    return text.gather(1, (lens - 1).long()[:, None])


def step_plain(model, text, lens):
    cu = torch.arange(model.B + 1, dtype=torch.int32, device=model.device)
    logits = spec_lmhead_logits(model.forward(last_tokens(text, lens).view(-1), cu), model.head)
    none = torch.zeros_like(lens)
    model.commit(text, lens, logits.argmax(1, keepdim=True).to(torch.int32), none)
    return none, logits


def step_chain(model, text, lens, K=4):
    drafts, _ = spec_prompt_lookup(text, lens, n_drafts=K)
    drafts.clamp_(min=0)  # what the text has no draft for is drafted as token 0
    cu = torch.arange(model.B + 1, dtype=torch.int32, device=model.device) * (K + 1)
    hidden = model.forward(torch.cat([last_tokens(text, lens), drafts], dim=1).view(-1), cu)
    need = spec_verify_lmhead_workspace_bytes(model.B, K, model.d, model.V)
    tokens, n = spec_verify_lmhead(hidden.view(model.B, K + 1, -1), model.head, None, drafts, mode="greedy",
                                   workspace=torch.empty(need, dtype=torch.uint8, device=model.device))
    model.commit(text, lens, tokens, n)
    return n, None


def step_tree(model, text, lens, K=4):
    """Two branches under the last token: the text's draft and, beside it, the
    draft after a shorter match."""
    B, dev = model.B, model.device
    first, _ = spec_prompt_lookup(text, lens, max_ngram=3, n_drafts=K)
    second, _ = spec_prompt_lookup(text, lens, max_ngram=1, n_drafts=K)
    nodes = torch.cat([last_tokens(text, lens), first.clamp(min=0), second.clamp(min=0)], dim=1)
    up = [-1, *range(K), 0, *range(K + 1, 2 * K)]
    parents = torch.tensor(up, dtype=torch.int32, device=dev).expand(B, -1).contiguous()
    N = 2 * K + 1
    cu = torch.arange(B + 1, dtype=torch.int32, device=dev) * N
    logits = spec_lmhead_logits(model.forward(nodes.view(-1), cu, parents), model.head)
    tokens, n, last = spec_verify_tree(logits.view(B, N, -1), nodes, parents)
    model.commit(text, lens, tokens, n, parents, last)
    return n, None


def step_sample(model, drafter, text, lens, uniforms, seed, K=4, **settings):
    """K tokens drawn from the drafter, one after another, and verified. uniforms
    [K, B] draw the drafts, seed the verify step's. settings: temperature, top_k,
    top_p, min_p, each a number or one per sequence ([B]). The drafter's cache takes the last draft too, so that whatever is
    kept is in it."""
    B, dev = model.B, model.device
    one = torch.arange(B + 1, dtype=torch.int32, device=dev)
    tokens, before, drafts, rows = last_tokens(text, lens), drafter.ctx, [], []
    for i in range(K + 1):
        logits = spec_lmhead_logits(drafter.forward(tokens.view(-1), one), drafter.head)
        drafter.ctx = drafter.ctx + 1
        if i < K:
            rows.append(spec_truncate_logits(logits, **settings))
            tokens = spec_sample(logits, uniforms[i], **settings)[:, None]
            drafts.append(tokens)
    drafts = torch.cat(drafts, dim=1)
    hidden = model.forward(torch.cat([last_tokens(text, lens), drafts], dim=1).view(-1), one * (K + 1))
    target = spec_lmhead_logits(hidden, model.head).view(B, K + 1, -1)
    spec_truncate_logits(target, **settings, out=target)
    temperature = settings.get("temperature", 1.0)
    if not torch.is_tensor(temperature):
        temperature = temperature or 1.0  # (a row cut at 0 has one token, likely at any temperature)
    out, n = spec_verify(target, torch.stack(rows, dim=1), drafts, temperature, "sample", seed)
    model.commit(text, lens, out, n)
    drafter.ctx = torch.minimum(before + 1 + n, lens - 1)
    return n, target


STEPS = {"plain": step_plain, "chain": step_chain, "tree": step_tree}


def example_prompts(B, V, seed=1):
    """Prompts that repeat themselves, so that there is something to look up."""
    g = torch.Generator().manual_seed(seed)
    return [torch.randint(0, V, (int(n),), generator=g).tolist() * 2 for n in torch.randint(4, 60, (B,), generator=g)]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--mode", choices=(*STEPS, "sample"), default="chain")
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--batch", type=int, default=8)
    a = ap.parse_args()
    L_max = 512
    kw = dict(score_cap=30.0, biased=True, pooled=True) if a.mode == "sample" else {}
    model = Decoder(a.batch, L_max, **kw)
    text, lens = start(model, example_prompts(a.batch, model.V), L_max)
    if a.mode == "sample":
        drafter = Decoder(a.batch, L_max, layers=1, **kw)
        start(drafter, example_prompts(a.batch, model.V), L_max)
    before = lens.clone()
    for i in range(a.steps):
        if a.mode == "sample":
            uniforms = torch.rand(4, a.batch, device=model.device)
            step_sample(model, drafter, text, lens, uniforms, i, temperature=0.8, top_k=40, top_p=0.9)
        else:
            STEPS[a.mode](model, text, lens)
    torch.cuda.synchronize()
    made = (lens - before).tolist()
    print(f"{a.mode}: {a.steps} steps, tokens per sequence and step {sum(made) / a.steps / a.batch:.2f} ({made})")


if __name__ == "__main__":
    main()
