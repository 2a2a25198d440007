"""Attention in fp16 where one key outweighs a long context, on the GPU against
the formula in 64 bits."""
import numpy as np
import pytest
import torch

from speculative_decoding_verification_24_gb300 import spec_paged_attention
from speculative_decoding_verification_24_gb300.build import build
from test_gpu_paged_attention import FP16, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("first_row", [0, 1])
def test_weights_far_below_the_largest_keep_their_sum(first_row):
    """The first key weighs about 2^26 times any other and its value is 0: the
    output is made of the small weights alone. As many sequences as CTAs, over
    the same pages: each CTA walks one of them alone. (first_row: one row tile,
    whose tiles two streams share, or two with a stream each.)

    A weight is rounded to fp16 with the largest of the row at 2^7 or above:
    half a step, 2^-11 of it or 2^-25 / 2^7 = 2^-32 of the largest. A score is
    a sum of D products in fp32 (error ds), sums take a step per 16 keys, and
    the output is rounded once (2^-11)."""
    dev, B, ctx, page, D = "cuda", torch.cuda.get_device_properties(0).multi_processor_count, 100000, 256, 64
    new = 200 if first_row else 1
    g = torch.Generator().manual_seed(4)
    pages = -(-(ctx + new) // page)
    k, v = torch.randn(pages * page, 1, D, generator=g) * 0.5, 1 + 0.1 * torch.randn(pages * page, 1, D, generator=g)
    k[0, 0, 0], v[0] = 18.5, 0.0
    k, v = (x.to(FP16).view(pages, page, 1, D) for x in (k, v))
    row = torch.randn(new, 1, D, generator=g) * 0.1
    row[:, :, 0] = 8.0  # the score is about the key's first element
    row, scale = row.to(FP16), 1 / 8
    table = torch.arange(pages, dtype=torch.int32).expand(B, -1).contiguous().to(dev)
    lens = torch.full((B,), ctx, dtype=torch.int32, device=dev)
    cu = (torch.arange(B + 1) * new).to(torch.int32).to(dev)
    lse = torch.empty(B * new, 1, device=dev)
    out = spec_paged_attention(row.repeat(B, 1, 1).to(dev), k.to(dev), v.to(dev), table, lens, cu, scale=scale, out_lse=lse)
    out, lse = out.view(B, new, D), lse.view(B, new)
    assert torch.equal(out, out[:1].expand_as(out)) and torch.equal(lse, lse[:1].expand_as(lse))
    kd, vd = k.double().view(-1, D), v.double().view(-1, D)
    for i in range(0, new, 67):
        n = ctx + i + 1
        q = row[i, 0].double()
        s = kd[:n] @ q * scale
        w = torch.exp(s - s.max())
        total = w.sum()
        want = w @ vd[:n] / total
        ds = float((kd[:n].abs() @ q.abs()).max()) * scale * (D + 8) * 2.0 ** -23
        held = torch.clamp(w * 2.0 ** -11, min=2.0 ** -32)
        bound = 1.01 * ((held @ vd[:n].abs()) / total + (2 * ds + (n / 16 + 16) * 2.0 ** -22 + 2.0 ** -11) * (w @ vd[:n].abs()) / total)
        assert (bound <= 0.06 * want.abs()).all()  # the small weights' sum is told from its parts
        err = (out[0, i].double().cpu() - want).abs()
        assert (err <= bound).all(), (i, float((err / bound).max()), float((err / want.abs()).max()))
        assert abs(float(lse[0, i]) - float(torch.logsumexp(s, 0))) <= ds + (n + 64) * 2.0 ** -24 + 2.0 ** -21 * (1 + float(s.max()))


def test_large_and_rising_scores_in_fp16():
    c = Case([(600, 3), (0, 140)], dtype=FP16, seed=9, q_scale=60.0)
    c.check(c.run())
    c = Case([(1500, 2), (900, 70)], Hq=4, Hkv=1, dtype=FP16, seed=10)
    for b in range(2):
        slots = np.arange(int(c.ctx[b] + c.cu[b + 1] - c.cu[b]))
        pages, at = torch.from_numpy(c.table[b, slots // 16].astype(np.int64)).cuda(), torch.from_numpy(slots % 16).cuda()
        c.k[pages, at] = (c.k[pages, at].float() * torch.from_numpy(0.02 * slots).cuda()[:, None, None]).to(FP16)
    c.check(c.run())
