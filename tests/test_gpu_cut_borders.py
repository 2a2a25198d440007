"""Cuts and draws whose goal lies next to a border: within 1e-11 of the sum, as the
interface says, they are those of the definition (cut_borders.py)."""
import numpy as np
import pytest
import torch

from cut_borders import Row

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def api():
    import speculative_decoding_verification_24_gb300 as sv
    return sv


def cuts(z, ps, **kw):
    """What is kept of the row z [V] for each top-p: masks [len(ps), V]."""
    ps = torch.as_tensor(np.asarray(ps, np.float32)).cuda()
    flags, n = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty(len(ps), dtype=torch.int32, device="cuda")
    out = api().spec_truncate_logits(z.cuda().expand(len(ps), -1), top_p=ps, out_n_kept=n, status_word=flags,
                                     out=torch.empty(len(ps), len(z), dtype=z.dtype, device="cuda"), **kw)
    kept = (out > float("-inf")).cpu().numpy()
    assert flags.item() == 0 and n.tolist() == kept.sum(1).tolist()
    return kept


def draws(z, us, **kw):
    us = torch.as_tensor(np.asarray(us, np.float32)).cuda()
    return api().spec_sample(z.cuda().expand(len(us), -1), us, **kw).tolist()


FAR = pytest.mark.parametrize("V,far,ps", [
    (200000, 25.0, (0.999999,)), (262144, 28.0, (1 - 2.0 ** -23,)), (250000, 22.5, (0.99998, 0.99999)), (262144, 22.0, (0.99995, 0.9999)),
    (3000, 24.0, (1 - 2.0 ** -23, 1 - 2.0 ** -24)), (40000, 20.0, (0.99999, 0.9999999)),
])


def far_below(V, far, dtype):
    z = torch.full((V,), -far).to(dtype)
    z[V // 3] = 0.0
    return z


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "fp32"))
@FAR
def test_many_equal_logits_far_below_the_first(dtype, V, far, ps):
    z = far_below(V, far, dtype)
    for k in (0, 1500):
        row = Row(z.double().numpy(), k=k)
        for p, kept in zip(ps, cuts(z, ps, top_k=k)):
            row.check_count(row.count_of(kept), p)


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "fp32"))
@FAR
def test_draws_from_many_equal_logits_far_below_the_first(dtype, V, far, ps):
    """Of all, of a list and of more than a list takes."""
    z = far_below(V, far, dtype)
    us = (0.5, 1 - 2.0 ** -24, 1 - 2.0 ** -22, 0.999999, 0.99999, 0.3)
    for k in (0, 1500, 2500, V - 7):
        if k < V:
            row = Row(z.double().numpy(), k=k)
            for u, token in zip(us, draws(z, us, top_k=k)):
                row.check_token(token, u)


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "fp32"))
@FAR
def test_many_equal_logits_below_a_large_top_k(dtype, V, far, ps):
    z = far_below(V, far, dtype)
    for k in (2500, V - 7):
        row = Row(z.double().numpy(), k=k)
        for p, kept in zip(ps, cuts(z, ps, top_k=k)):
            row.check_count(row.count_of(kept), p)


def usual(V, dtype, sigma, seed):
    z = (torch.randn(V, generator=torch.Generator().manual_seed(seed)) * sigma).to(dtype)
    if seed % 2:
        z[seed % V] = z.float().max() + 3 * sigma  # a few tokens hold most
        z[(7 * seed) % V] = z.float().max() - sigma
    return z


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "fp32"))
@pytest.mark.parametrize("V,sigma,T", ((2000, 3.0, 1.0), (5000, 3.0, 0.8), (5000, 1.0, 1.0), (32000, 2.0, 1.3), (151936, 1.5, 1.0), (151936, 3.0, 0.7)))
def test_draws_next_to_an_edge(dtype, V, sigma, T):
    checked = 0
    for seed in (1, 2, 3, 4):
        z = usual(V, dtype, sigma, seed)
        row = Row(z.double().numpy(), T)
        us = row.near_draws(64)
        checked += len(us)
        if len(us):
            for x, token in zip(us, draws(z, us, temperature=T)):
                row.check_token(token, x)
        # of what a large top-k leaves
        k = V - V // 5
        row = Row(z.double().numpy(), T, k)
        us = row.near_draws(32)
        checked += len(us)
        if len(us):
            for x, token in zip(us, draws(z, us, temperature=T, top_k=k)):
                row.check_token(token, x)
    assert checked > 50


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "fp32"))
@pytest.mark.parametrize("V,sigma,T", ((5000, 3.0, 0.8), (5000, 0.5, 1.0), (32000, 1.0, 1.3), (151936, 1.0, 1.0), (151936, 1.5, 1.0), (262144, 0.3, 1.0)))
def test_cuts_next_to_a_border(dtype, V, sigma, T):
    checked = 0
    for seed in (2, 3, 4):
        z = usual(V, dtype, sigma, seed)
        for k in (0, 3000, V - V // 5):
            if k and k >= V:
                continue
            row = Row(z.double().numpy(), T, k)
            ps = row.near_cuts(48)
            checked += len(ps)
            if not len(ps):
                continue
            kept = cuts(z, ps, temperature=T, top_k=k)
            for p, x in zip(ps, kept):
                row.check_count(row.count_of(x), p)
            # and a draw of what is kept, next to an edge of it
            n = row.count_of(kept[0])
            us = row.near_draws(4, n=n)
            if len(us):
                for u, token in zip(us, draws(z, us, temperature=T, top_k=k, top_p=float(ps[0]))):
                    row.check_token(token, u, n)
    assert checked > 30


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "fp32"))
def test_short_lists_next_to_a_border(dtype):
    """top-k of up to 2048: sums in a list."""
    checked = 0
    for seed, V, sigma, k in ((1, 5000, 2.0, 50), (2, 32000, 2.0, 128), (3, 32000, 1.0, 129), (4, 5000, 0.3, 1500), (6, 32000, 0.2, 2048),
                              (8, 151936, 0.5, 2000), (10, 151936, 0.3, 1024)):
        z = usual(V, dtype, sigma, seed)
        row = Row(z.double().numpy(), 0.9, k)
        ps = row.near_cuts(40, most=2e-9)
        if len(ps):
            for p, kept in zip(ps, cuts(z, ps, temperature=0.9, top_k=k)):
                row.check_count(row.count_of(kept), p)
                checked += 1
        us = row.near_draws(40, most=2e-9)
        if len(us):
            for u, token in zip(us, draws(z, us, temperature=0.9, top_k=k)):
                row.check_token(token, u)
                checked += 1
    assert checked > 20


@pytest.mark.parametrize("offset", (2.0 ** 15, -2.0 ** 15))
def test_a_maximum_without_room_for_float_sums(offset):
    """256 log2(e) max / T above 2^21: every weight is formed in whole units."""
    z = usual(50000, F32, 2.0, 2) + offset
    row = Row(z.double().numpy())
    us, ps = row.near_draws(40), row.near_cuts(40)
    for u, token in zip(us, draws(z, us)):
        row.check_token(token, u)
    for p, kept in zip(ps, cuts(z, ps)):
        row.check_count(row.count_of(kept), p)
    assert len(us) + len(ps) > 20


@pytest.mark.parametrize("offset,T", ((0.0, 1.0), (7.3, 0.7), (-90.0, 1.3), (400.0, 0.9)))
def test_draws_next_to_an_edge_of_few_tokens(offset, T):
    """Rows of 5 tokens, two of which hold most: the error of a single weight counts
    whole. Of a million such rows those where some u lies next to an edge."""
    g = torch.Generator().manual_seed(int(abs(offset)))
    z = torch.randn(1_000_000, 5, generator=g) - 4.0
    z[:, 1] = 0.0
    z[:, 3] = -torch.rand(len(z), generator=g) * 3.0
    z = z * T + offset
    zd = z.double().numpy()
    w = np.exp((zd - zd.max(1, keepdims=True)) / np.float64(np.float32(T)))
    sums = w.cumsum(1)
    edges = sums[:, 1] / sums[:, -1]  # (right to 1e-15)
    u = edges.astype(np.float32)
    gap = u.astype(np.float64) - edges
    rows = np.nonzero((np.abs(gap) > 1.2e-11) & (np.abs(gap) < 2e-10))[0]
    assert len(rows) > 2000
    tokens = api().spec_sample(z[rows].cuda(), torch.from_numpy(u[rows]).cuda(), temperature=T).cpu().numpy()
    # below the edge it is the token before it, else one behind it
    assert np.array_equal(tokens <= 1, gap[rows] < 0), f"{int(((tokens <= 1) != (gap[rows] < 0)).sum())} of {len(rows)}"
