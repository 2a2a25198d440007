"""spec_sample and spec_truncate_logits against the definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

from cut_reference import cut_row, draw

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
BAD_ROW, BAD_SETTING = 2, 1024


def api():
    import speculative_decoding_verification_24_gb300 as sv
    return sv


def rows_of(n, V, dtype, seed, sigma=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, V, generator=g) * sigma).to(dtype)


def value(x, b):
    return x[b].item() if torch.is_tensor(x) else (0 if x is None else x)


def check(logits, u, settings, R=1, out=None, placed=None):
    """Both operators over logits [N, V] (host), as they lie in `placed` (device,
    [B, V] or [B, R, V]). Returns how many rows lay too near a border to tell."""
    sv = api()
    N, V = logits.shape
    dev = logits.cuda() if placed is None else placed
    if R > 1 and placed is None:
        dev = dev.view(N // R, R, V)
    on = {n: x.cuda() if torch.is_tensor(x) else x for n, x in settings.items()}
    logprobs, count = torch.full(dev.shape[:-1], 7.0, device="cuda"), torch.zeros(dev.shape[:-1], dtype=torch.int32, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    tokens = sv.spec_sample(dev, u.cuda().view(dev.shape[:-1]), **on, out_logprobs=logprobs, status_word=flags)
    cut = sv.spec_truncate_logits(dev, **on, out=out, out_n_kept=count, status_word=flags)
    torch.cuda.synchronize()
    tokens, logprobs, count = tokens.view(-1).tolist(), logprobs.view(-1).tolist(), count.view(-1).tolist()
    cut = cut.float().cpu().reshape(N, V).numpy()
    z64, want_flags, unclear = logits.double().numpy(), 0, 0
    for i in range(N):
        f = lambda n, d: (settings[n][i // R].item() if torch.is_tensor(settings.get(n)) else  # noqa: E731
                          np.float32(settings.get(n, d)).item() if settings.get(n, d) is not None else d)
        T, k, p, m = f("temperature", 1.0), int(f("top_k", 0)), f("top_p", 1.0), f("min_p", 0.0)
        ref = cut_row(z64[i], T, k, p, m)
        if ref is None:
            top = z64[i].max()
            want_flags |= (BAD_ROW if not math.isfinite(top) else 0)
            if not (T == 0 or 2.0 ** -64 <= T <= 2.0 ** 64) or k < 0 or not 0 <= p <= 1 or not 0 <= m <= 1:
                want_flags |= BAD_SETTING
            assert tokens[i] == -1 and math.isnan(logprobs[i]) and count[i] == -1
            assert np.array_equal(cut[i], logits[i].float().numpy(), equal_nan=True)
            continue
        keep, w, near = ref
        if near:
            unclear += 1
            continue
        assert np.array_equal(cut[i], np.where(keep, logits[i].float().numpy(), -np.inf)), i
        assert count[i] == keep.sum()
        token, logprob, near = draw(keep, w, u.view(-1)[i].item())
        if near:
            unclear += 1
            continue
        assert tokens[i] == token, i
        # the sum is right to 2^-32, the logarithm is rounded once
        if math.isfinite(logprob):
            assert abs(logprobs[i] - logprob) <= 2.0 ** -24 * abs(logprob) + 2.0 ** -31, i
    assert flags.item() == want_flags
    return unclear


SETTINGS = [
    dict(), dict(temperature=0.7, top_k=50, top_p=0.9), dict(top_p=0.95), dict(top_k=1), dict(min_p=0.05), dict(temperature=0.0),
    dict(temperature=1.5, top_k=300), dict(top_k=1500, top_p=0.99), dict(top_k=2000), dict(top_p=0.5, min_p=0.01),
    dict(temperature=0.3, top_p=0.999), dict(top_p=0.0), dict(min_p=1.0), dict(top_k=40, top_p=0.8, min_p=0.1), dict(top_p=1e-6),
]


@pytest.mark.parametrize("settings", SETTINGS, ids=str)
@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "fp32"))
def test_settings(settings, dtype):
    unclear = 0
    for V in (2, 3, 7, 33, 1000, 4099, 32000):
        n = 6 if V < 5000 else 3
        u = torch.rand(n, generator=torch.Generator().manual_seed(V))
        unclear += check(rows_of(n, V, dtype, V), u, settings)
    assert unclear <= 1


@pytest.mark.parametrize("dtype,V", ((BF16, 151936), (F32, 128256), (F32, 262144), (BF16, 262144), (BF16, 200001), (F32, 99999)))
def test_long_rows(dtype, V):
    """Every way that a row can take, several CTAs per row."""
    logits = rows_of(len(SETTINGS), V, dtype, 5, sigma=2.0)
    per = lambda name, d, dt: torch.tensor([s.get(name, d) for s in SETTINGS], dtype=dt)  # noqa: E731
    settings = dict(temperature=per("temperature", 1.0, F32), top_k=per("top_k", 0, torch.int32), top_p=per("top_p", 1.0, F32),
                    min_p=per("min_p", 0.0, F32))
    u = torch.rand(len(SETTINGS), generator=torch.Generator().manual_seed(V))
    assert check(logits, u, settings) <= 1


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "fp32"))
@pytest.mark.parametrize("V", (5, 700, 5000, 150001))
def test_equal_logits(dtype, V):
    """Ties go by index; more of them than any list takes."""
    flat = torch.full((8, V), -3.25).to(dtype)
    two = flat.clone()
    two[:, ::3] = 0.5
    signs = torch.zeros(8, V).to(dtype)
    signs[:, 1::2] = -0.0  # equal to 0
    ks = torch.tensor([0, 1, 2, V // 3, V // 2, V - 1, V, V + 5], dtype=torch.int32)
    u = torch.tensor([0.0, 0.3, 0.5, 0.9999999, 0.25, 0.75, 0.999, 0.1])
    for z in (flat, two, signs):
        check(z, u, dict(top_k=ks))
        check(z, u, dict(top_p=torch.tensor([0.5, 0.25, 0.75, 0.125, 0.0, 1.0, 0.999, 0.1])))
        check(z, u, dict(top_k=ks, top_p=0.5, temperature=0.5))
        check(z, u, dict(temperature=0.0))
        check(z, u, dict(min_p=0.5))


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "fp32"))
def test_infinities_and_few_finite(dtype):
    z = rows_of(9, 3000, dtype, 1)
    z[0, 5:] = -math.inf                  # 5 finite ones
    z[1, ::2] = -math.inf
    z[2, :] = -math.inf                   # none
    z[3, 77] = math.nan
    z[4, 2999] = math.inf
    z[5, :2999] = -math.inf               # the last alone
    z[6, 1000:] = -math.inf
    z[7] = torch.where(torch.arange(3000) % 7 == 0, z[7].float(), -math.inf).to(dtype)
    u = torch.linspace(0, 0.99, 9)
    for s in (dict(), dict(top_k=20), dict(top_k=2000), dict(top_k=1200, top_p=0.9), dict(top_p=0.99), dict(min_p=0.2),
              dict(temperature=0.0), dict(top_k=2999, min_p=1e-30)):
        assert check(z, u, s) <= 1


@pytest.mark.parametrize("scale", (1e-30, 1e-3, 1e3, 1e30))
def test_magnitudes(scale):
    z = rows_of(6, 4001, F32, 3) * scale
    u = torch.linspace(0.05, 0.95, 6)
    for T in (2.0 ** -60, min(max(0.01 * scale, 2.0 ** -64), 2.0 ** 64), 1.0, 1e4, 2.0 ** 60):
        for s in (dict(top_k=30), dict(top_p=0.9), dict(min_p=0.3), dict()):
            check(z, u, dict(temperature=T, **s))


def test_a_far_offset_keeps_its_differences():
    """Logits near 1000 that differ by single steps of fp32."""
    z = 1000.0 + torch.arange(64, dtype=F32)[None, torch.randperm(64, generator=torch.Generator().manual_seed(0))] * 2.0 ** -14
    check(z.expand(4, 64).contiguous(), torch.tensor([0.1, 0.4, 0.6, 0.9]), dict(temperature=2.0 ** -12, top_p=0.9))


def test_uniforms_at_and_past_the_ends():
    z = rows_of(6, 500, F32, 8)
    u = torch.tensor([0.0, -1.0, math.nan, 1.0 - 2.0 ** -24, 1.0, 5.0])
    check(z, u, dict())
    check(z, u, dict(top_k=7))


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "fp32"))
def test_the_end_of_a_row_whose_weights_hardly_count(dtype):
    """u of 1 and next to it where the last tokens' weights are below any unit but
    their sum is not: a token that can be drawn comes out all the same."""
    sv = api()
    for V, far in ((20000, 34.0), (150000, 36.0), (20000, 60.0), (3000, 800.0)):
        z = torch.full((4, V), -far).to(dtype)
        z[:, 5] = 0.0
        z[1, V // 2:] = -math.inf
        u = torch.tensor([1.0, 1.0, 1.0 - 2.0 ** -24, 2.0]).cuda()
        lp = torch.empty(4, device="cuda")
        for kw in (dict(), dict(top_p=0.99999), dict(top_k=2500)):
            tokens = sv.spec_sample(z.cuda(), u, **kw, out_logprobs=lp).tolist()
            for i, t in enumerate(tokens):
                assert 0 <= t < V and z[i, t] > -math.inf, (V, far, kw, i)
            assert tokens[2] == 5


def test_settings_per_sequence_and_out_of_range():
    B, R, V = 14, 3, 900
    z = rows_of(B * R, V, F32, 2)
    z[5, 3] = math.nan
    T = torch.tensor([1, 0, 0.5, -1, math.nan, math.inf, 1, 1, 1, 1, 1, 1, 2.0 ** -70, 2.0])
    k = torch.tensor([0, 9, 40, 1, 1, 1, -1, 5, 5, 5, 0, 0, 3, 2000], dtype=torch.int32)
    p = torch.tensor([0.9, 1, 1, 1, 1, 1, 1, -0.1, 1.5, math.nan, 1, 1, 1, 0.7])
    m = torch.tensor([0, 0, 0.01, 0, 0, 0, 0, 0, 0, 0, -0.5, math.nan, 0, 0])
    u = torch.rand(B * R, generator=torch.Generator().manual_seed(4))
    check(z, u, dict(temperature=T, top_k=k, top_p=p, min_p=m), R=R)


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "fp32"))
def test_strides_and_alignment(dtype):
    """Rows that begin anywhere; outputs laid out and aligned unlike them, in
    place, and with what lies between the rows left alone."""
    B, R = 3, 2
    for V, shift in ((1001, 1), (4096, 3), (77, 5), (15, 7), (8, 1), (50003, 2)):
        z = rows_of(B * R, V, dtype, V)
        u = torch.rand(B * R, generator=torch.Generator().manual_seed(V))
        big = torch.full((B + 1, R + 2, V + 13), 3.0, dtype=dtype, device="cuda")
        placed = big[:B, 1:1 + R, shift:shift + V]
        placed.copy_(z.view(B, R, V))
        before = big.clone()
        check(z, u, dict(top_k=11, top_p=0.9), R=R, placed=placed)
        other = torch.full((R, B + 1, V + 9), 5.0, dtype=dtype, device="cuda")
        out = other[:, :B, 2:2 + V].transpose(0, 1)
        check(z, u, dict(top_p=0.8), R=R, placed=placed, out=out)
        left = other.clone()
        left[:, :B, 2:2 + V] = 5.0
        assert torch.equal(left, torch.full_like(left, 5.0))
        assert torch.equal(big, before)
        check(z, u, dict(temperature=0.8, min_p=0.1), R=R, placed=placed, out=placed)
        big[:B, 1:1 + R, shift:shift + V] = before[:B, 1:1 + R, shift:shift + V]
        assert torch.equal(big, before)


def test_a_row_read_by_all_sequences():
    """A stride of 0: one row of logits, many draws."""
    z = rows_of(1, 5000, F32, 6)
    placed = z.cuda().expand(40, 5000)
    check(z.expand(40, 5000).contiguous(), torch.linspace(0, 0.999, 40), dict(top_k=25), placed=placed, out=torch.empty(40, 5000, device="cuda"))


def test_many_rows_and_repeats():
    """More clusters than the GPU holds at once; the same bits every time."""
    sv = api()
    z = rows_of(700, 9001, BF16, 9, sigma=2.0)
    T = torch.tensor([0.0, 0.7, 1.0, 1.0])[torch.arange(700) % 4]
    k = torch.tensor([0, 40, 1200], dtype=torch.int32)[torch.arange(700) % 3]
    p = torch.tensor([1.0, 0.9])[torch.arange(700) // 3 % 2]
    u = torch.rand(700, generator=torch.Generator().manual_seed(1))
    assert check(z, u, dict(temperature=T, top_k=k, top_p=p)) <= 2
    dev = [x.cuda() for x in (z, u, T, k, p)]
    runs = []
    for _ in range(5):
        lp = torch.empty(700, device="cuda")
        tok = sv.spec_sample(dev[0], dev[1], temperature=dev[2], top_k=dev[3], top_p=dev[4], out_logprobs=lp)
        cut = sv.spec_truncate_logits(dev[0], temperature=dev[2], top_k=dev[3], top_p=dev[4])
        runs.append((tok, lp, cut))
    for r in runs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(r, runs[0]))


def test_draws_follow_the_distribution():
    """Frequencies over a grid of u are the probabilities, to one step of it."""
    sv = api()
    n, V = 20000, 37
    z = rows_of(1, V, F32, 4, sigma=1.5)
    u = ((torch.arange(n) + 0.5) / n).cuda()
    tokens = sv.spec_sample(z.cuda().expand(n, V), u, temperature=0.9, top_k=20, top_p=0.95)
    keep, w, _ = cut_row(z[0].double().numpy(), np.float32(0.9).item(), 20, np.float32(0.95).item(), 0.0)
    want = np.where(keep, w, 0) / w[keep].sum()
    got = torch.bincount(tokens.long(), minlength=V).double().cpu().numpy() / n
    assert np.abs(got - want).max() <= 1.01 / n


def test_graph_and_stream():
    sv = api()
    z = [rows_of(5, 6000, F32, s).cuda() for s in (1, 2)]
    u = torch.rand(5, generator=torch.Generator().manual_seed(3)).cuda()
    want = [(sv.spec_sample(x, u, top_k=30), sv.spec_truncate_logits(x, top_p=0.9)) for x in z]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    live, tok, cut = z[0].clone(), torch.empty(5, dtype=torch.int32, device="cuda"), torch.empty_like(z[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_sample(live, u, top_k=30, out_tokens=tok)
        sv.spec_truncate_logits(live, top_p=0.9, out=cut)
    for x, (t, c) in zip(z[::-1], want[::-1]):
        live.copy_(x)
        graph.replay()
        assert torch.equal(tok, t) and torch.equal(cut, c)
    with torch.cuda.stream(stream):
        t = sv.spec_sample(z[1], u, top_k=30)
    t2 = sv.spec_sample(z[1], u, top_k=30, stream=stream)
    torch.cuda.current_stream().wait_stream(stream)
    assert torch.equal(t, want[1][0]) and torch.equal(t2, want[1][0])


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "fp32"))
def test_drafts_drawn_cut_and_verified(dtype):
    """As a decoder uses them: drafts drawn from the draft's cut rows, both
    models' rows cut, verified. What comes out lies in the target's cut, and a
    draft's probabilities are those of the cut rows."""
    sv = api()
    B, K, V, T = 24, 4, 8000, 0.8
    target = rows_of(B * (K + 1), V, dtype, 11, sigma=2.0).view(B, K + 1, V).cuda()
    noise = torch.randn(B, K, V, generator=torch.Generator().manual_seed(12)).cuda()
    draft = (target[:, :K].float() + 0.5 * noise).to(dtype)
    u = torch.rand(B, K, generator=torch.Generator().manual_seed(13)).cuda()
    settings = dict(temperature=T, top_k=60, top_p=0.9)
    lp = torch.empty(B, K, device="cuda")
    drafts = sv.spec_sample(draft, u, **settings, out_logprobs=lp)
    cut_d, cut_t = sv.spec_truncate_logits(draft, **settings), sv.spec_truncate_logits(target, **settings)
    full = sv.spec_verify_ex(cut_t, cut_d, drafts, T, seed=7, debug=True)
    n, tokens = full["n_accepted"].tolist(), full["tokens"].tolist()
    assert min(n) >= 0 and max(n) > 0
    p_draft = torch.softmax(cut_d.double() / np.float32(T).item(), -1).gather(2, drafts.long()[..., None])[..., 0]
    # 2^-20: the verify step's probabilities are right to 1e-5 / 10 here; log in fp32
    assert ((lp.double() - p_draft.log()).abs() <= 2.0 ** -20 * (1 + lp.abs())).all()
    for b in range(B):
        for i in range(n[b] + 1):
            assert cut_t[b, i, tokens[b][i]].item() > -math.inf


@pytest.mark.parametrize("seed", range(12))
def test_random_shapes_and_settings(seed):
    """Rows of any length and spread, as they lie in a padded buffer, with settings
    per sequence or one for all."""
    g = torch.Generator().manual_seed(100 + seed)
    pick = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))  # noqa: E731
    B, R = pick(1, 6), pick(1, 4)
    V = int(2 ** (1 + 16 * torch.rand(1, generator=g).item()))
    V, dtype = max(2, V), (BF16, F32)[seed % 2]
    z = (torch.randn(B * R, V, generator=g) * 10.0 ** (torch.rand(B * R, 1, generator=g) * 2 - 1)).to(dtype)
    row, seq = V + pick(0, 9), 0
    seq = R * row + pick(0, 9)
    flat = torch.full((B * seq + 16,), math.nan, dtype=dtype, device="cuda")
    placed = torch.as_strided(flat, (B, R, V), (seq, row, 1), pick(0, 8))
    placed.copy_(z.view(B, R, V))
    any_of = lambda *x: x[pick(0, len(x) - 1)]  # noqa: E731
    make = dict(temperature=lambda: any_of(0.0, 0.2, 0.7, 1.0, 3.0), top_k=lambda: any_of(0, 1, 5, 50, 700, V, V - 1),
                top_p=lambda: any_of(0.0, 0.3, 0.9, 0.99, 1.0, 1.0), min_p=lambda: any_of(0.0, 0.0, 0.02, 0.5))
    settings = {}
    for name, one in make.items():
        if pick(0, 1):
            settings[name] = torch.tensor([one() for _ in range(B)], dtype=torch.int32 if name == "top_k" else F32)
        else:
            settings[name] = one()
    assert check(z, torch.rand(B * R, generator=g), settings, R=R, placed=placed) <= 1


@pytest.mark.parametrize("offset", (3.0, 12.0, 100.0))
def test_the_largest_weight_is_one_wherever_the_maximum_lies(offset):
    """256 log2(e) max / T next to halves of whole numbers too."""
    g = torch.Generator().manual_seed(int(offset))
    z = torch.randn(6000, 16, generator=g) + offset * (0.5 + torch.rand(6000, 1, generator=g))
    assert check(z, torch.rand(6000, generator=g), dict()) <= 1
