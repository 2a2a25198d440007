"""Paged attention with capped scores and a bias by distance against the formula
in 64 bits."""
import math

import numpy as np
import pytest
import torch

from paged_reference import HALF_STEP, SMALLEST, entries, make_cache, make_table, path_to, visible
from speculative_decoding_verification_24_gb300 import spec_paged_attention, spec_paged_attention_workspace
from speculative_decoding_verification_24_gb300.build import build

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def usual_slopes(Hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], dtype=torch.float32)


def position(ctx, i, parents):
    if parents is None:
        return ctx + i
    path = path_to(parents, i)
    return ctx if path is None else ctx + len(path) - 1


class Case:
    """A batch: seqs is a list of (context, new tokens)."""

    def __init__(self, seqs, Hq=8, Hkv=2, D=128, page=16, dtype=BF16, parents=None, seed=0, q_scale=3.0, cap=0.0, slopes=None,
                 dirty=True):
        g, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
        self.seqs, self.Hq, self.Hkv, self.D, self.page, self.dtype = seqs, Hq, Hkv, D, page, dtype
        self.ctx = np.array([c for c, _ in seqs], np.int32)
        self.cu = np.concatenate([[0], np.cumsum([n for _, n in seqs])]).astype(np.int32)
        need = [-(-(c + n) // page) for c, n in seqs]
        pages = sum(need) + 3
        self.k, self.v = make_cache(pages, page, Hkv, D, dtype, g)
        self.table = make_table(need, pages, rng)
        if dirty:  # entries behind each sequence's last token hold anything
            used = np.zeros((pages, page), bool)
            for b, (c, n) in enumerate(seqs):
                slots = np.arange(c + n)
                used[self.table[b, slots // page], slots % page] = True
            junk = torch.from_numpy(~used).cuda()
            for x, bad in ((self.k, float("nan")), (self.v, float("inf"))):
                x.masked_fill_(junk[:, :, None, None], bad)
        self.q = (torch.randn(int(self.cu[-1]), Hq, D, generator=g) * q_scale).to(dtype).cuda()
        self.cap, self.slopes, self.parents, self.scale = cap, slopes, parents, D ** -0.5
        self.args = [torch.from_numpy(x).cuda() for x in (self.table, self.ctx, self.cu)]
        self.tree = None if parents is None else torch.from_numpy(parents).cuda()

    def run(self, **kw):
        self.lse = torch.full((self.q.shape[0], self.Hq), float("nan"), device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        kw.setdefault("score_cap", self.cap or None)
        kw.setdefault("bias_slopes", None if self.slopes is None else self.slopes.cuda())
        out = spec_paged_attention(self.q, self.k, self.v, *self.args, scale=self.scale, tree_parents=self.tree, out_lse=self.lse,
                                   status_word=self.status, **kw)
        torch.cuda.synchronize()
        return out

    def reference(self):
        """Output, lse and the bounds of their errors. Beside those of the plain
        scores (paged_reference.attention) a capped score is off by 2^-21 of the
        cap, an added bias by the fp32 roundings of slope, product and sum: 3 of
        half a step each, of magnitudes at most |bias| + |score|; a score error ds
        moves a weight by at most 2 ds of itself. Only scores that matter count:
        what lies 40 below the row's largest has weight e^-40 whatever its error
        of less than 1 is."""
        T, Hq, D, u = self.q.shape[0], self.Hq, self.D, HALF_STEP[self.dtype]
        G = Hq // self.Hkv
        qd = self.q.cpu().double()
        out, bound = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, D, dtype=torch.float64)
        lse, lse_bound = torch.full((T, Hq), -math.inf, dtype=torch.float64), torch.zeros(T, Hq, dtype=torch.float64)
        for b, (ctx, n) in enumerate(self.seqs):
            if n == 0:
                continue
            par = None if self.parents is None else self.parents[b]
            k, v = (entries(x, self.table, b, range(ctx + n), self.page) for x in (self.k, self.v))
            where = np.array(list(range(ctx)) + [position(ctx, i, par) for i in range(n)], np.float64)
            for i in range(n):
                seen = visible(ctx, i, par)
                if not seen:
                    continue
                t = int(self.cu[b]) + i
                ks, vs = k[seen].transpose(0, 1), v[seen].transpose(0, 1)
                qs = qd[t].reshape(self.Hkv, G, D)
                s = qs @ ks.transpose(1, 2) * self.scale
                ds = (qs.abs() @ ks.abs().transpose(1, 2) * self.scale) * (D + 8) * 2.0 ** -23
                if self.cap:
                    s = self.cap * torch.tanh(s / self.cap)
                    ds = ds + self.cap * 2.0 ** -21  # (tanh's slope is at most 1)
                if self.slopes is not None:
                    bias = self.slopes.double().view(self.Hkv, G, 1) * torch.from_numpy(where[seen] - position(ctx, i, par))
                    ds = ds + 3 * 2.0 ** -24 * (bias.abs() + s.abs())
                    s = s + bias
                matter = s > s.amax(-1, keepdim=True) - 40
                ds = torch.where(matter, ds, 0.0).amax(-1)
                w = torch.softmax(s, dim=-1)
                o, a = w @ vs, w @ vs.abs()
                rel = u + 2 * ds[..., None] + (len(seen) / 16 + 16) * 2.0 ** -22
                out[t] = o.reshape(Hq, D)
                bound[t] = 1.01 * (rel * a + u * o.abs() + u * rel * a).reshape(Hq, D) + SMALLEST[self.dtype]
                lse[t] = torch.logsumexp(s, dim=-1).reshape(Hq)
                lse_bound[t] = (ds + (len(seen) + 64) * 2.0 ** -24).reshape(Hq) + 2.0 ** -21 * (1 + lse[t].abs())
        return out, bound, lse, lse_bound

    def check(self, out=None, status=0):
        out = self.run() if out is None else out
        assert int(self.status) == status
        ref, bound, lse, lse_bound = self.reference()
        err = (out.double().cpu() - ref).abs()
        assert torch.isfinite(out).all()
        worst = (err / bound.clamp(min=1e-300)).max() if err.numel() else 0.0
        assert (err <= bound).all(), f"{float(worst):.2f} times the bound, max error {float(err.max()):.3g}"
        got = self.lse.double().cpu()
        none = torch.isinf(lse)
        assert torch.equal(torch.isinf(got), none)
        assert ((got - lse).abs() <= lse_bound)[~none].all()


KINDS = {"cap": dict(cap=20.0), "bias": dict(slopes=True), "both": dict(cap=8.0, slopes=True)}


def kind(name, Hq):
    k = dict(KINDS[name])
    if k.get("slopes"):
        k["slopes"] = usual_slopes(Hq)
    return k


SMALL = [(0, 1), (5, 1), (127, 1), (128, 1), (126, 3), (300, 5), (0, 7), (40, 0), (255, 2), (1500, 1)]


@pytest.mark.parametrize("name", list(KINDS))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 2), (7, 1)])
def test_single_tokens_and_drafts(name, D, dtype, Hq, Hkv):
    Case(SMALL, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, seed=D + Hq, **kind(name, Hq)).check()


@pytest.mark.parametrize("name", list(KINDS))
@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, FP16)])
@pytest.mark.parametrize("Hq,Hkv,seqs", [
    (8, 2, [(0, 31), (0, 32), (0, 33), (0, 65), (0, 129)]), (4, 4, [(0, 127), (3, 128), (0, 129), (500, 257)]),
    (14, 2, [(0, 18), (1, 19), (200, 36), (300, 55)]), (128, 1, [(0, 1), (130, 2), (20, 5)]),
])
def test_chunks(name, D, dtype, Hq, Hkv, seqs):
    Case(seqs, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, seed=Hq, **kind(name, Hq)).check()


@pytest.mark.parametrize("name", list(KINDS))
@pytest.mark.parametrize("page", [8, 24, 128, 1000])
def test_page_sizes(name, page):
    Case([(0, 3), (777, 4), (130, 1), (1030, 9)], page=page, D=64, seed=page, **kind(name, 8)).check()


@pytest.mark.parametrize("name", list(KINDS))
def test_one_context_over_all_ctas(name):
    Case([(40000, 3)], Hq=4, Hkv=1, seed=6, **kind(name, 4)).check()


def trees(B, N, seed):
    rng = np.random.default_rng(seed)
    par = np.full((B, N), -1, np.int32)
    for b in range(B):
        for i in range(1, N):
            par[b, i] = rng.integers(max(0, i - 4), i)
    return par


@pytest.mark.parametrize("name", list(KINDS))
@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, FP16)])
def test_trees(name, D, dtype):
    """A node's distance goes by depths; contexts that put the nodes on both
    sides of a tile's edge; a broken tree's nodes see nothing."""
    ctx = [0, 1, 100, 120, 127, 128, 250, 400]
    par = trees(len(ctx), 32, 4)
    seqs = [(c, 32 if i % 2 else 19) for i, c in enumerate(ctx)]
    Case(seqs, D=D, dtype=dtype, parents=par, seed=7, **kind(name, 8)).check()
    par[3, 5] = 9
    Case(seqs, D=D, dtype=dtype, parents=par, seed=7, **kind(name, 8)).check(status=128)


def test_scores_past_the_cap_and_infinite():
    """Scores of many times the cap bend to it; infinite ones are the cap."""
    c = Case([(300, 2), (50, 40)], q_scale=200.0, cap=3.0, seed=8, dirty=False)
    c.check()
    c = Case([(200, 3)], Hq=2, Hkv=1, cap=5.0, seed=9, dirty=False)
    c.q[:, :, 0] = 30000.0
    c.k[..., 0] = 0.0
    at = [int(x) for x in (c.table[0, 20 // 16], 20 % 16)]
    c.k[at[0], at[1], 0, 0] = float("inf")
    out = c.run()
    ref = c.q.new_tensor(0)
    k, v = (entries(x, c.table, 0, range(203), 16) for x in (c.k, c.v))
    for i in range(3):
        s = (c.q[i].cpu().double() @ k[:203 - 2 + i, 0].T) * c.scale
        ref = torch.softmax(5.0 * torch.tanh(s / 5.0), -1) @ v[:203 - 2 + i, 0]
        assert (out[i].cpu().double() - ref).abs().max() < 0.05  # half a step of weights and values of at most 4: 2^-8 * 4 * 2


def test_slopes_of_either_sign_zero_and_far():
    slopes = torch.tensor([0.0, -0.01, 1.0, 30.0, 1e-6, -1e-3, 0.5, 2.0 ** -8])
    Case([(700, 3), (129, 30), (5000, 1)], slopes=slopes, seed=10).check()
    # (a weight of the last key alone)
    Case([(700, 3)], slopes=torch.full((8,), 1000.0), seed=11).check()


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_a_cap_that_does_nothing_and_slopes_of_zero(dtype):
    """A large cap and zero slopes give what the plain call gives, within the
    change's own error."""
    c = Case([(300, 1), (77, 4), (0, 60)], dtype=dtype, q_scale=1.0, seed=12, cap=4096.0, slopes=torch.zeros(8))
    c.check()
    changed, plain = c.run(), c.run(score_cap=None, bias_slopes=None)
    assert (changed.double() - plain.double()).abs().max() <= 2.0 ** -6


@pytest.mark.parametrize("name", list(KINDS))
def test_repeats_graph_and_workspace(name):
    c = Case([(3000, 1), (500, 4), (4000, 9)], seed=13, **kind(name, 8))
    ws = spec_paged_attention_workspace(14, 8, 2, 128)
    first = c.run(workspace=ws)
    for _ in range(3):
        assert torch.equal(c.run(workspace=ws), first)
    out = torch.empty_like(first)
    graph = torch.cuda.CUDAGraph()
    slopes = None if c.slopes is None else c.slopes.cuda()
    with torch.cuda.graph(graph):
        spec_paged_attention(c.q, c.k, c.v, *c.args, scale=c.scale, out=out, workspace=ws, score_cap=c.cap or None, bias_slopes=slopes)
    for _ in range(2):
        out.zero_()
        graph.replay()
        assert torch.equal(out, first)


def test_values_that_are_not_finite():
    """As in the plain call, such a value reaches the tokens that see it only."""
    c = Case([(200, 30)], cap=10.0, slopes=usual_slopes(8), seed=14, dirty=False)
    want = c.run()
    page, at = int(c.table[0, 210 // 16]), 210 % 16
    c.v[page, at, 0, 5] = float("inf")
    out = c.run()
    assert torch.isfinite(out[:10]).all() and torch.equal(out[:10], want[:10])
    assert (out[10:, :4, 5] == float("inf")).all()
    assert torch.equal(out[10:, 4:], want[10:, 4:])


@pytest.mark.parametrize("power", (-60, 60))
def test_the_smallest_and_largest_scale_of_a_cap(power):
    """At 2^-60 all keys that a token sees count alike; at 2^60 scores are the cap,
    minus it or 0. Masked and unread entries stay out of both."""
    c = Case([(300, 3), (0, 40), (128, 1)], cap=4.0, seed=15)
    c.scale = 4.0 * 2.0 ** power
    g = torch.Generator().manual_seed(16)
    c.q = torch.randint(-1, 2, c.q.shape, generator=g).to(BF16).cuda()
    fill = torch.randint(-1, 2, c.k.shape, generator=g).to(BF16).cuda()
    c.k = torch.where(torch.isnan(c.k), c.k, fill)  # products are whole numbers, of up to 128: exact
    out = c.run()
    for b, (ctx, n) in enumerate(c.seqs):
        k, v = (entries(x, c.table, b, range(ctx + n), c.page) for x in (c.k, c.v))
        for i in range(n):
            t, seen = int(c.cu[b]) + i, ctx + i + 1
            s = torch.einsum("hgd,shd->hgs", c.q[t].cpu().double().view(2, 4, 128), k[:seen].double())
            w = torch.softmax(4.0 * torch.sign(s) if power > 0 else torch.zeros_like(s), -1)
            ref = torch.einsum("hgs,shd->hgd", w, v[:seen].double()).reshape(8, 128)
            size = torch.einsum("hgs,shd->hgd", w, v[:seen].double().abs()).reshape(8, 128)
            # weights and output are rounded by half a step each; scores are off by 2^-21 of the cap
            assert ((out[t].cpu().double() - ref).abs() <= 1.01 * (2.0 ** -8 + 2.0 ** -17) * size + 2.0 ** -8 * ref.abs()).all()


@pytest.mark.parametrize("name", list(KINDS))
@pytest.mark.parametrize("D", [64, 128])
def test_results_do_not_depend_on_what_ran_before(name, D):
    """Scores that no row sees are what the memory held: large ones of another
    call, or none. Neither they nor the entries behind the last token count."""
    c = Case([(5, 1), (100, 5), (300, 2), (0, 40), (700, 1)], D=D, seed=17, dirty=False, q_scale=0.3, **kind(name, 8))
    other = Case([(900, 130)] * 8, D=D, seed=18, q_scale=300.0, **kind(name, 8))
    first, lse = c.run(), c.lse
    rows = torch.arange(c.k.shape[0] * c.page, device="cuda").view(-1, c.page)
    used = torch.zeros_like(rows, dtype=torch.bool)
    for b, (ctx, n) in enumerate(c.seqs):
        at = torch.arange(ctx + n)
        used[torch.from_numpy(c.table)[b, at // c.page].long().cuda(), (at % c.page).cuda()] = True
    for junk in (0.0, 1e4, float("nan"), None):
        other.run()
        if junk is not None:
            c.k.masked_fill_(~used[:, :, None, None], junk)
        assert torch.equal(c.run(), first) and torch.equal(c.lse, lse)
