"""A bias by distance over contexts of tens of millions of keys, beyond the whole
numbers that fp32 holds. The table names a few pages again and again."""
import pytest
import torch

from paged_reference import HALF_STEP, SMALLEST
from speculative_decoding_verification_24_gb300 import spec_paged_attention
from speculative_decoding_verification_24_gb300.build import build

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("cap", (None, 20.0))
@pytest.mark.parametrize("dtype", (BF16, FP16), ids=("bf16", "fp16"))
@pytest.mark.parametrize("ctx,n,tree", ((40_000_001, 3, False), (33_554_432 + 77, 1, False), (70_000_000, 5, True), (16_777_300, 2, False)))
def test_bias_over_far_keys(ctx, n, tree, dtype, cap):
    """Slopes below 0 put the weight on the farthest keys, small ones on all."""
    build()
    D, page, Hq = 64, 65536, 4
    slopes = torch.tensor([-2.0 ** -10, -3e-4, 2.0 ** -22, -1e-7], device="cuda")
    g = torch.Generator("cuda").manual_seed(ctx % 1000 + n)
    k, v = (torch.randn(3, page, 1, D, generator=g, device="cuda").to(dtype) for _ in range(2))
    pages = -(-(ctx + n) // page)
    table = (torch.arange(pages, device="cuda") * 7 % 3).to(torch.int32)[None]
    q = torch.randn(n, Hq, D, generator=g, device="cuda").to(dtype)
    parents = [-1] + [i // 2 for i in range(n - 1)]
    ctx_t, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([ctx], [0, n]))
    lse = torch.empty(n, Hq, device="cuda")
    out = spec_paged_attention(q, k, v, table, ctx_t, cu, scale=D ** -0.5, score_cap=cap, bias_slopes=slopes, out_lse=lse,
                               tree_parents=torch.tensor([parents], dtype=torch.int32, device="cuda") if tree else None)
    at = torch.arange(ctx + n, device="cuda")
    entry = table[0].long()[at // page] * page + at % page
    kd, vd = k.double().view(-1, D), v.double().view(-1, D)
    for i in range(n):
        path = [i]
        while tree and path[-1] > 0:
            path.append(parents[path[-1]])
        depth = len(path) - 1 if tree else i
        position = at.double()
        if tree:  # a node's position goes by its depth
            for j in range(n):
                p, d = j, 0
                while p > 0:
                    p, d = parents[p], d + 1
                position[ctx + j] = ctx + d
        seen = at < ctx if tree else at <= ctx + i
        if tree:
            seen[[ctx + j for j in path]] = True
        for h in range(Hq):
            s = (kd @ q[i, h].double()) * D ** -0.5
            ds = (kd.abs() @ q[i, h].double().abs()).max() * D ** -0.5 * (D + 8) * 2.0 ** -23
            if cap:
                s = cap * torch.tanh(s / cap)
                ds = ds + cap * 2.0 ** -21
            bias = slopes[h].double() * (position - (ctx + depth))
            score = torch.where(seen, s[entry] + bias, float("-inf"))
            top = score.max()
            matter = score > top - 40
            ds = ds + 3 * 2.0 ** -24 * (bias.abs() + s[entry].abs())[matter].max()
            w = torch.exp(score - top)
            total = w.sum()
            # weights by entry of the three pages
            per = torch.zeros(3 * page, dtype=torch.float64, device="cuda").index_add_(0, entry, w / total)
            ref, size = per @ vd, per @ vd.abs()
            u = HALF_STEP[dtype]
            # (fp32 sums over a thread's keys, of which each CTA has 1 of about 150)
            many = float(matter.sum())
            rel = u + 2 * float(ds) + (many / 150 / 16 + 16) * 2.0 ** -22
            err = (out[i, h].double() - ref).abs()
            bound = 1.01 * (rel * size + u * ref.abs() + u * rel * size) + SMALLEST[dtype]
            assert (err <= bound).all(), (i, h, float((err / bound).max()))
            exact = float(top + total.log())
            assert abs(float(lse[i, h]) - exact) <= float(ds) + (many / 150 + 64) * 2.0 ** -24 + 2.0 ** -21 * (1 + abs(exact)), (i, h)
