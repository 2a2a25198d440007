"""Attention over the paged cache on the GPU against the formula in 64 bits."""
import numpy as np
import pytest
import torch

from paged_reference import attention, make_cache, make_table, path_to
from speculative_decoding_verification_24_gb300 import binding, spec_paged_attention, spec_paged_attention_workspace
from speculative_decoding_verification_24_gb300.build import build

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


class Case:
    """A batch: seqs is a list of (context, new tokens)."""

    def __init__(self, seqs, Hq=8, Hkv=2, D=128, page=16, dtype=BF16, layout="tokens", parents=None, seed=0, q_scale=2.0,
                 spare=3, dirty=True):
        g, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
        self.ctx = np.array([c for c, _ in seqs], np.int32)
        self.cu = np.concatenate([[0], np.cumsum([n for _, n in seqs])]).astype(np.int32)
        self.page, self.D, self.Hkv, self.Hq, self.parents = page, D, Hkv, Hq, parents
        need = [-(-(c + n) // page) for c, n in seqs]
        self.k, self.v = make_cache(sum(need) + spare, page, Hkv, D, dtype, g, layout)
        self.table = make_table(need, sum(need) + spare, rng)
        if dirty:  # entries behind each sequence's last token, and free pages, hold anything
            used = np.zeros((sum(need) + spare, page), bool)
            for b, (c, n) in enumerate(seqs):
                slots = np.arange(c + n)
                used[self.table[b, slots // page], slots % page] = True
            junk = torch.from_numpy(~used).cuda()
            for x, bad in ((self.k, float("nan")), (self.v, float("inf"))):
                x.masked_fill_(junk[:, :, None, None], bad)
        self.q = (torch.randn(int(self.cu[-1]), Hq, D, generator=g) * q_scale).to(dtype).cuda()
        self.scale = D ** -0.5
        self.args = [torch.from_numpy(x).cuda() for x in (self.table, self.ctx, self.cu)]
        self.tree = None if parents is None else torch.from_numpy(parents).cuda()

    def run(self, **kw):
        self.lse = torch.full((self.q.shape[0], self.Hq), float("nan"), device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        kw.setdefault("q", self.q)
        kw.setdefault("scale", self.scale)
        kw.setdefault("status_word", self.status)
        out = spec_paged_attention(kw.pop("q"), self.k, self.v, *self.args, tree_parents=self.tree, out_lse=self.lse, **kw)
        torch.cuda.synchronize()
        return out

    def check(self, out, status=0):
        assert int(self.status) == status
        ref, bound, lse, lse_bound = attention(self.q, self.k, self.v, self.table, self.ctx, self.cu, self.page, self.scale,
                                               self.parents)
        err = (out.double().cpu() - ref).abs()
        assert torch.isfinite(out).all()
        worst = (err / bound.clamp(min=1e-300)).max() if err.numel() else 0.0
        assert (err <= bound).all(), f"{float(worst):.2f} times the bound, max error {float(err.max()):.3g}"
        got = self.lse.double().cpu()
        none = torch.isinf(lse)
        assert torch.equal(torch.isinf(got), none)
        assert ((got - lse).abs() <= lse_bound)[~none].all()


SMALL = [(0, 1), (5, 1), (127, 1), (128, 1), (126, 3), (300, 5), (0, 7), (40, 0), (255, 2)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 2), (7, 1), (6, 2)])
def test_single_tokens_and_drafts(D, dtype, Hq, Hkv):
    c = Case(SMALL, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, seed=D + Hq)
    c.check(c.run())


def test_one_token_of_one_sequence():
    for ctx in (0, 1, 15, 127, 128, 129, 1000):
        c = Case([(ctx, 1)], seed=ctx)
        c.check(c.run())


@pytest.mark.parametrize("page", [8, 16, 24, 48, 64, 128, 256, 1000])
def test_page_sizes(page):
    c = Case([(0, 3), (777, 4), (130, 1), (1030, 9)], page=page, D=64, seed=page)
    c.check(c.run())


@pytest.mark.parametrize("layout", ["tokens", "heads", "halves"])
def test_cache_layouts(layout):
    c = Case([(100, 3), (250, 40), (0, 1)], layout=layout, page=32, seed=3)
    c.check(c.run())


@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, FP16)])
@pytest.mark.parametrize("Hq,Hkv,seqs", [
    (8, 2, [(0, 31), (0, 32), (0, 33), (0, 64), (0, 65), (0, 129)]),       # tile and pair edges (32 tokens a tile)
    (4, 4, [(0, 127), (3, 128), (0, 129), (500, 256), (7, 257)]),          # one head a row: 128 tokens a tile
    (14, 2, [(0, 18), (1, 19), (200, 36), (0, 37), (300, 55)]),            # 7 heads: 18 tokens a tile, 2 rows over
    (128, 1, [(0, 1), (130, 2), (20, 5)]),                                 # 128 heads: a token a tile
    (100, 1, [(0, 2), (300, 3)]),                                          # 100 heads: 28 rows of each tile unused
])
def test_chunks(D, dtype, Hq, Hkv, seqs):
    c = Case(seqs, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, seed=Hq)
    c.check(c.run())


def test_prompt_and_decoding_in_one_batch():
    c = Case([(400, 1), (0, 300), (1000, 5), (64, 150), (2000, 1)], Hq=8, Hkv=2, seed=5)
    c.check(c.run())


def test_one_long_context_over_all_ctas():
    c = Case([(40000, 9)], Hq=4, Hkv=1, D=128, seed=6)
    c.check(c.run())


@pytest.mark.parametrize("Hq,D,new", [(2, 64, 2), (3, 128, 1), (1, 128, 200)])
def test_long_shares(Hq, D, new):
    # a score of tiles per CTA: every stage of the pipeline is used many times
    rng = np.random.default_rng(21)
    seqs = [(int(rng.integers(6000, 12000)), new) for _ in range(45 if new < 10 else 6)]
    c = Case(seqs, Hq=Hq, Hkv=1, D=D, page=16, seed=21, dirty=False)
    c.check(c.run())


def test_long_chunk_cut_into_pieces():
    c = Case([(5000, 70)], Hq=4, Hkv=1, D=64, seed=7)
    c.check(c.run())


def test_many_short_sequences():
    rng = np.random.default_rng(8)
    seqs = [(int(rng.integers(0, 40)), int(rng.integers(0, 3))) for _ in range(900)]
    c = Case(seqs, Hq=2, Hkv=1, D=64, page=8, seed=8)
    c.check(c.run())


def test_large_scores_keep_the_softmax_in_range():
    c = Case([(600, 3), (0, 140)], seed=9, q_scale=60.0)
    c.check(c.run())


def test_rising_scores_raise_the_maximum_in_every_tile():
    # keys grow along the context, so that later tiles dominate all before them
    c = Case([(1500, 2), (900, 70)], Hq=4, Hkv=1, seed=10)
    for b in range(2):
        slots = np.arange(int(c.ctx[b] + c.cu[b + 1] - c.cu[b]))
        pages, at = torch.from_numpy(c.table[b, slots // 16].astype(np.int64)).cuda(), torch.from_numpy(slots % 16).cuda()
        c.k[pages, at] = (c.k[pages, at].float() * torch.from_numpy(0.02 * slots).cuda()[:, None, None]).to(BF16)
    c.check(c.run())


def random_tree(n, N, rng, chain=0.3):
    p = np.full(N, -1, np.int32)
    for i in range(1, n):
        p[i] = i - 1 if rng.random() < chain else rng.integers(0, i)
    return p


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (16, 2, 64), (3, 3, 64)])
def test_trees(Hq, Hkv, D):
    rng = np.random.default_rng(11)
    seqs = [(0, 32), (100, 32), (120, 20), (127, 9), (500, 1), (3, 31), (96, 32)]
    c = Case(seqs, Hq=Hq, Hkv=Hkv, D=D, parents=np.stack([random_tree(n, 32, rng) for _, n in seqs]), seed=11)
    c.check(c.run())


def test_nodes_of_a_broken_tree_see_nothing():
    rng = np.random.default_rng(12)
    parents = np.stack([random_tree(12, 12, rng, chain=1.0) for _ in range(3)])
    parents[1, 4] = 9      # not an earlier node: nodes 4.. of the chain see nothing
    parents[2, 1] = -1
    c = Case([(50, 12)] * 3, parents=parents, seed=12)
    out = c.run()
    c.check(out, status=binding.SV_FLAG_BAD_TREE)
    assert (out[12 + 4:24] == 0).all() and torch.isinf(c.lse[12 + 4:24]).all()
    assert (out[12:12 + 4] != 0).any()


def test_strided_queries_and_output():
    c = Case([(90, 3), (0, 70), (300, 1)], Hq=8, Hkv=2, D=64, seed=13)
    T = c.q.shape[0]
    fused = torch.randn(T, 8 + 4, 64, device="cuda").to(BF16)
    fused[:, 2:10] = c.q
    wide = torch.full((8, T, 64), 7.0, dtype=BF16, device="cuda")
    out = c.run(q=fused[:, 2:10], out=wide.transpose(0, 1))
    assert out.data_ptr() == wide.data_ptr()
    c.check(out)


def test_page_table_of_a_larger_batch():
    c = Case([(90, 3), (40, 7)], seed=14)
    big = torch.full((5, c.table.shape[1] + 4), -5, dtype=torch.int32, device="cuda")
    big[1::2, :c.table.shape[1]] = c.args[0]
    c.args[0] = big[1::2, :c.table.shape[1]]
    c.check(c.run())


def test_rows_no_sequence_claims_are_left_alone():
    c = Case([(90, 3), (40, 7)], seed=15)
    q = torch.cat([c.q, torch.full((4, 8, 128), float("nan"), dtype=BF16, device="cuda")])
    out = torch.full_like(q, 5.0)
    lse = torch.full((14, 8), 5.0, device="cuda")
    spec_paged_attention(q, c.k, c.v, *c.args, out=out, out_lse=lse)
    torch.cuda.synchronize()
    assert (out[10:] == 5).all() and (lse[10:] == 5).all()
    assert torch.equal(out[:10], c.run())


def test_no_rows_at_all():
    c = Case([(90, 3)], seed=16)
    args = [c.args[0], c.args[1], torch.zeros(2, dtype=torch.int32, device="cuda")]
    out = spec_paged_attention(c.q[:0], c.k, c.v, *args)
    assert out.shape == (0, 8, 128)
    out = torch.full_like(c.q, 3.0)  # rows, but of no sequence
    spec_paged_attention(c.q, c.k, c.v, *args, out=out)
    torch.cuda.synchronize()
    assert (out == 3).all()


def test_bad_lengths_and_pages_are_flagged():
    c = Case([(90, 3), (40, 7), (20, 2), (33, 1)], seed=17, dirty=False)
    good = c.run()
    room = c.table.shape[1] * c.page
    ctx = c.args[1].clone()
    ctx[0], ctx[2] = -1, room - 1  # negative; one entry too many
    c.args[1], keep = ctx, c.args[1]
    out = c.run()
    assert int(c.status) == binding.SV_FLAG_BAD_LENGTH
    assert (out[:3] == 0).all() and (out[10:12] == 0).all()
    assert torch.isinf(c.lse[:3]).all() and torch.isinf(c.lse[10:12]).all()
    assert torch.equal(out[3:10], good[3:10]) and torch.equal(out[12:], good[12:])
    c.args[1] = keep
    # rows out of [0, T), or descending, belong to nobody
    cu = c.args[2].clone()
    cu[1], cu[2] = 10, 3
    c.args[2], keep = cu, c.args[2]
    out = c.run(out=torch.full_like(c.q, 2.0))
    assert int(c.status) == binding.SV_FLAG_BAD_LENGTH and (out == 2).all()
    c.args[2] = keep
    # a page that is not there reads as zeros: scores 0, values 0
    table = c.args[0].clone()
    table[1, 1] = -3
    table[3, 0] = c.k.shape[0]
    c.args[0], kept = table, c.args[0]
    out = c.run()
    assert int(c.status) == binding.SV_FLAG_BAD_PAGE
    assert torch.equal(out[:3], good[:3]) and torch.equal(out[10:12], good[10:12])
    zeroed = Case([(90, 3), (40, 7), (20, 2), (33, 1)], seed=17, dirty=False)
    for b, j in ((1, 1), (3, 0)):
        zeroed.k[int(kept[b, j])] = 0
        zeroed.v[int(kept[b, j])] = 0
    assert torch.equal(out, zeroed.run())


def test_overlapping_sequences_are_refused():
    # every other sequence claims all rows: more work than any valid call has
    T, B = 3000, 1000
    c = Case([(5, 1)], Hq=2, Hkv=1, D=64, seed=23)
    q = torch.randn(T, 2, 64, device="cuda").to(BF16)
    cu = torch.tensor([T * (b % 2) for b in range(B + 1)], dtype=torch.int32, device="cuda")
    table = torch.zeros(B, 4000, dtype=torch.int32, device="cuda")
    out, status = torch.full_like(q, 2.0), torch.zeros(1, dtype=torch.int32, device="cuda")
    spec_paged_attention(q, c.k, c.v, table, torch.full((B,), 50000, dtype=torch.int32, device="cuda"), cu, out=out,
                         status_word=status)
    torch.cuda.synchronize()
    assert int(status) == binding.SV_FLAG_BAD_LENGTH and (out == 2).all()


def test_what_is_not_finite_stays_with_the_rows_that_see_it():
    c = Case([(200, 6), (30, 4)], Hq=4, Hkv=2, seed=24)
    want = c.run()
    q = c.q.clone()
    q[2, 1], q[7, 3] = float("nan"), float("inf")
    out = c.run(q=q)
    lost = torch.zeros(10, 4, dtype=torch.bool, device="cuda")
    lost[2, 1] = lost[7, 3] = True
    assert torch.equal(torch.isnan(out).any(-1), lost) and torch.equal(out[~lost], want[~lost])
    # a key of the chunk: the tokens before it do not see it
    slot = 203
    c.k[int(c.table[0, slot // 16]), slot % 16, 1] = float("nan")
    out = c.run()
    lost[:] = False
    lost[3:6, 2:] = True
    assert torch.equal(torch.isnan(out).any(-1), lost) and torch.equal(out[~lost], want[~lost])


def test_calls_repeat_bit_for_bit_and_leave_the_workspace_ready():
    c = Case([(3000, 5), (100, 200), (0, 1), (900, 33)], Hq=8, Hkv=2, seed=18)
    ws = spec_paged_attention_workspace(c.q.shape[0], 8, 2, 128)
    first, lse = c.run(workspace=ws), c.lse
    c.check(first)
    for _ in range(20):
        assert torch.equal(c.run(workspace=ws), first) and torch.equal(c.lse, lse)
    assert (ws[:binding.SV_PAGED_WORKSPACE_HEAD] == 0).all()
    # whatever the rest of the workspace holds
    ws[binding.SV_PAGED_WORKSPACE_HEAD:].fill_(0xFF)
    assert torch.equal(c.run(workspace=ws), first)


def test_another_stream_and_a_graph():
    c = Case([(3000, 5), (100, 70)], seed=19)
    want = c.run()
    ws = spec_paged_attention_workspace(c.q.shape[0], 8, 2, 128)
    side = torch.cuda.Stream()
    out = torch.zeros_like(c.q)
    torch.cuda.synchronize()
    spec_paged_attention(c.q, c.k, c.v, *c.args, out=out, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        spec_paged_attention(c.q, c.k, c.v, *c.args, out=out, workspace=ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    # the graph reads lengths and tables when it runs
    c.args[1].copy_(torch.tensor([2500, 50], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, c.run())


def test_a_wait_that_gives_up_is_flagged():
    c = Case([(3000, 5), (100, 70)], seed=20)
    want = c.run()
    ws = spec_paged_attention_workspace(c.q.shape[0], 8, 2, 128)
    c.run(workspace=ws, flags=binding.SV_ARG_TEST_WAIT_TIMEOUT)
    assert int(c.status) & binding.SV_FLAG_TIMEOUT
    ws[:binding.SV_PAGED_WORKSPACE_HEAD].zero_()
    assert torch.equal(c.run(workspace=ws), want)
    assert int(c.status) == 0


@pytest.mark.parametrize("seqs,Hq,Hkv,D,dtype,tree", [
    ([(200, 6), (30, 4), (125, 9)], 4, 2, 128, BF16, False),     # one tile of rows, tiles that the chunk straddles
    ([(0, 9), (119, 9), (40, 1)], 8, 2, 64, FP16, False),
    ([(60000, 9)], 8, 1, 128, BF16, False),                      # many pieces
    ([(900, 20), (2000, 30)], 8, 2, 64, BF16, False),            # few
    ([(0, 700), (3, 130), (1000, 300)], 8, 2, 128, BF16, False),   # two tiles of rows
    ([(250, 1000)], 32, 1, 128, FP16, False),                    # row tiles of 4 tokens, cut
    ([(100, 32), (30, 32), (0, 17)], 8, 2, 128, BF16, True),
    ([(5000, 32), (96, 32)], 16, 2, 64, FP16, True),
])
def test_a_value_that_is_not_finite_stays_with_the_rows_that_see_it(seqs, Hq, Hkv, D, dtype, tree):
    rng = np.random.default_rng(5)
    parents = None
    if tree:
        parents = np.array([[int(rng.integers(max(0, i - 6), i)) if i else 0 for i in range(32)] for _ in seqs], np.int32)
    c = Case(seqs, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, parents=parents, seed=31)
    ref, bound, lse, lse_bound = attention(c.q, c.k, c.v, c.table, c.ctx, c.cu, c.page, c.scale, c.parents)
    G = Hq // Hkv
    extra = torch.zeros_like(ref)  # what the planted values add to the rows that see them
    bad = [float("inf"), -float("inf"), float("nan"), float("inf")]
    for b, (ctx, n) in enumerate(seqs):
        for x in range(min(n, 4)):
            node, h = int(rng.integers(0, n)), int(rng.integers(0, Hkv))
            slot = ctx + node
            at = (int(c.table[b, slot // 16]), slot % 16, h)
            for col in rng.permutation(D)[:3].tolist():
                if not np.isfinite(float(c.v[at][col])):
                    continue
                c.v[at][col] = bad[x]
                for i in range(node, n):
                    if not tree or node in path_to(parents[b], i):
                        extra[int(c.cu[b]) + i, h * G:(h + 1) * G, col] += bad[x]
    got = c.run().double().cpu()
    assert int(c.status) == 0
    clean = extra == 0
    assert clean.any() and not clean.all()
    assert ((got - ref).abs() <= bound)[clean].all()
    assert torch.equal(got[~clean].nan_to_num(7.0, 8.0, 9.0), extra[~clean].nan_to_num(7.0, 8.0, 9.0))
    assert ((c.lse.double().cpu() - lse).abs() <= lse_bound).all()


def test_nodes_of_a_broken_tree_see_nothing_whatever_the_context_holds():
    parents = np.array([[0, 0, 5, 2, 1, 0]], np.int32)  # nodes 2 and 3 hang on nothing
    c = Case([(300, 6)], parents=parents, seed=32)
    c.v[int(c.table[0, 1]), 3] = float("nan")
    out = c.run()
    assert int(c.status) == binding.SV_FLAG_BAD_TREE
    assert (out[2:4] == 0).all() and torch.isneginf(c.lse[2:4]).all()
    assert torch.isnan(out[[0, 1, 4, 5]]).all()


@pytest.mark.parametrize("Hq,value", [(8, float("nan")), (64, float("inf"))])
def test_nodes_of_a_broken_tree_see_nothing_of_a_root_without_context(Hq, value):
    parents = np.array([[0, 0, 5, 2, 1, 0]], np.int32)
    c = Case([(0, 6)], Hq=Hq, parents=parents, seed=33)
    c.v[int(c.table[0, 0]), 0] = value
    out = c.run()
    assert int(c.status) == binding.SV_FLAG_BAD_TREE
    assert (out[2:4] == 0).all() and torch.isneginf(c.lse[2:4]).all()
    assert (out[[0, 1, 4, 5]].isfinite() == 0).all()


def test_rows_written_by_other_lanes_take_what_is_not_finite():
    # two row tiles, whole, full: a row's pieces are stored by the lanes of its
    # group and read back by its own
    c = Case([(0, 64)] * 200, Hq=4, Hkv=1, D=128, seed=34, dirty=False)
    want = c.run().clone()
    col = torch.arange(0, 128, 9, device="cuda")
    at = torch.from_numpy(c.table[:, 2]).cuda().long()  # slot 40 of each sequence
    c.v[at[:, None], 8, 0, col] = float("inf")
    out = c.run().view(200, 64, 4, 128)
    seen = torch.zeros_like(out, dtype=torch.bool)
    seen[:, 40:, :, col] = True
    assert (out[seen] == float("inf")).all()
    assert torch.equal(out[:, :40], want.view(200, 64, 4, 128)[:, :40])
    assert torch.isfinite(out[~seen]).all()


@pytest.mark.parametrize("kw,error", [
    (dict(workspace=torch.zeros(1 << 24, dtype=torch.uint8)), "workspace must live"),
    (dict(out_lse=torch.zeros(3, 8)), "out_lse must live"),
    (dict(status_word=torch.zeros(1, dtype=torch.int32)), "status_word must live"),
    (dict(status_word=torch.zeros(0, dtype=torch.int32)), "no element"),
    (dict(status_word=torch.zeros(1)), "int32"),
])
def test_tensors_that_do_not_belong_are_refused(kw, error):
    c = Case([(20, 3)], seed=35)
    with pytest.raises((ValueError, TypeError), match=error):
        spec_paged_attention(c.q, c.k, c.v, *c.args, **kw)


def test_an_item_that_takes_over_a_second():
    # little more than an item of 190 million keys per CTA (one page, read again
    # and again): the next item's queries wait for as long as the first one runs,
    # about 3 * 10^9 cycles
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    page, pages, T, D = 65536, 2900, 2 * (sms + 8), 64
    g = torch.Generator("cuda").manual_seed(36)
    k, v = (torch.randn(1, page, 1, D, generator=g, device="cuda").to(BF16) for _ in range(2))
    q = torch.randn(T, 128, D, generator=g, device="cuda").to(BF16)
    table = torch.zeros(1, pages, dtype=torch.int32, device="cuda")
    lens = torch.tensor([(pages - 1) * page], dtype=torch.int32, device="cuda")
    cu, status = torch.tensor([0, T], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = spec_paged_attention(q, k, v, table, lens, cu, status_word=status)
    torch.cuda.synchronize()
    assert int(status) == 0 and torch.isfinite(out).all()


@pytest.mark.parametrize("Hq,D,dtype", [(8, 64, FP16), (14, 128, FP16), (8, 128, BF16)])
def test_items_of_few_pieces_repeat_bit_for_bit(Hq, D, dtype):
    # a hundred items cut in two or three, joined by whichever CTA ends last:
    # either warpgroup's columns, and the lse, come out the same
    rng = np.random.default_rng(37)
    c = Case([(int(rng.integers(500, 2500)), 5) for _ in range(70)], Hq=Hq, Hkv=2, D=D, dtype=dtype, seed=37, dirty=False)
    ws = spec_paged_attention_workspace(c.q.shape[0], Hq, 2, D)
    first, lse = c.run(workspace=ws), c.lse
    for _ in range(300):
        assert torch.equal(c.run(workspace=ws), first) and torch.equal(c.lse, lse)
