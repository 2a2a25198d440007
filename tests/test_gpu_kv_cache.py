"""Appending to the paged cache and keeping a tree's path in it, on the GPU
against the definitions in 64 bits."""
import numpy as np
import pytest
import torch

from paged_reference import make_cache, make_table, path_to, rotate, rotate_bound
from speculative_decoding_verification_24_gb300 import binding, rope_inv_freq, spec_kv_append, spec_kv_commit
from speculative_decoding_verification_24_gb300.build import build

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


class Batch:
    def __init__(self, seqs, Hq=4, Hkv=2, D=128, page=16, dtype=BF16, layout="tokens", seed=0):
        g, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
        self.seqs, self.page, self.dtype = seqs, page, dtype
        self.ctx = np.array([c for c, _ in seqs], np.int32)
        self.cu = np.concatenate([[0], np.cumsum([n for _, n in seqs])]).astype(np.int32)
        need = [-(-(c + n) // page) for c, n in seqs]
        self.k_cache, self.v_cache = make_cache(sum(need) + 2, page, Hkv, D, dtype, g, layout)
        self.table = make_table(need, sum(need) + 2, rng)
        T = int(self.cu[-1])
        qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(dtype).cuda()
        self.q, self.k, self.v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        self.args = [torch.from_numpy(x).cuda() for x in (self.table, self.ctx, self.cu)]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def append(self, **kw):
        out = spec_kv_append(self.k, self.v, self.k_cache, self.v_cache, *self.args, status_word=self.status, **kw)
        torch.cuda.synchronize()
        return out

    def check(self, before, q_in, q_out, inv_freq, interleaved=False, parents=None, positions=None):
        k_ref, v_ref = (x.cpu().double() for x in before)
        k_bound = torch.zeros_like(k_ref)
        q_in, k_in, v_in = q_in.cpu().double(), self.k.cpu().double(), self.v.cpu()
        f = np.zeros(0) if inv_freq is None else inv_freq.numpy()
        for b, (ctx, n) in enumerate(self.seqs):
            for i in range(n):
                t, slot = int(self.cu[b]) + i, ctx + i
                pos = slot if parents is None else ctx + len(path_to(parents[b], i)) - 1
                pos = pos if positions is None else int(positions[t])
                at = (int(self.table[b, slot // self.page]), slot % self.page)
                value, mag = rotate(k_in[t], pos, f, interleaved)
                k_ref[at], k_bound[at], v_ref[at] = value, rotate_bound(value, mag, self.dtype), v_in[t].double()
                value, mag = rotate(q_in[t], pos, f, interleaved)
                assert ((q_out[t].cpu().double() - value).abs() <= rotate_bound(value, mag, self.dtype)).all()
        assert torch.equal(self.v_cache.cpu().double(), v_ref)
        assert ((self.k_cache.cpu().double() - k_ref).abs() <= k_bound).all()  # 0 where nothing was stored
        assert int(self.status) == 0


SEQS = [(0, 1), (15, 1), (16, 3), (0, 0), (100, 5), (0, 40), (47, 2)]


@pytest.mark.parametrize("D,rotary", [(128, 128), (128, 32), (64, 64), (64, 48), (128, 0)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(D, rotary, dtype, interleaved):
    b = Batch(SEQS, D=D, dtype=dtype, seed=D + rotary)
    before = b.k_cache.clone(), b.v_cache.clone()
    f = rope_inv_freq(rotary) if rotary else None
    q_out = b.append(q=b.q, inv_freq=f, interleaved=interleaved)
    b.check(before, b.q, q_out, f, interleaved)


@pytest.mark.parametrize("layout,page", [("heads", 8), ("halves", 64), ("tokens", 24)])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (7, 1), (3, 3), (16, 8)])
def test_append_layouts(layout, page, Hq, Hkv):
    b = Batch(SEQS, Hq=Hq, Hkv=Hkv, D=64, layout=layout, page=page, seed=Hq)
    before = b.k_cache.clone(), b.v_cache.clone()
    f = rope_inv_freq(64, 500000.0)
    b.check(before, b.q, b.append(q=b.q, inv_freq=f), f)


def test_append_many_tokens():
    # more tokens than CTAs take one at a time, sequences of every small length
    b = Batch([(i % 5, i % 4) for i in range(700)], Hq=2, Hkv=1, D=64, page=8, seed=2)
    before = b.k_cache.clone(), b.v_cache.clone()
    f = rope_inv_freq(64)
    b.check(before, b.q, b.append(q=b.q, inv_freq=f), f)


def test_append_tree_takes_depths():
    rng = np.random.default_rng(3)
    seqs = [(20, 12), (0, 1), (33, 7)]
    parents = np.full((3, 12), -1, np.int32)
    for b, (_, n) in enumerate(seqs):
        for i in range(1, n):
            parents[b, i] = rng.integers(0, i)
    b = Batch(seqs, seed=3)
    before = b.k_cache.clone(), b.v_cache.clone()
    f = rope_inv_freq(128)
    q_out = b.append(q=b.q, inv_freq=f, tree_parents=torch.from_numpy(parents).cuda())
    b.check(before, b.q, q_out, f, parents=parents)


def test_append_far_and_negative_positions():
    b = Batch([(3, 6)], Hq=2, Hkv=1, seed=4)
    pos = np.array([2 ** 31 - 1, -(2 ** 31), 10 ** 6, 131071, -7, 2 ** 24 + 1], np.int32)
    before = b.k_cache.clone(), b.v_cache.clone()
    f = rope_inv_freq(128)
    q_out = b.append(q=b.q, inv_freq=f, positions=torch.from_numpy(pos).cuda())
    b.check(before, b.q, q_out, f, positions=pos)


def test_append_in_place_and_without_queries():
    b, c = Batch(SEQS, seed=5), Batch(SEQS, seed=5)
    f = rope_inv_freq(128)
    want = b.append(q=b.q, inv_freq=f)
    assert c.append(q=c.q, q_out=c.q, inv_freq=f) is c.q
    assert torch.equal(c.q, want) and torch.equal(c.k_cache, b.k_cache)
    d = Batch(SEQS, seed=5)
    assert d.append(inv_freq=f) is None
    assert torch.equal(d.k_cache, b.k_cache) and torch.equal(d.v_cache, b.v_cache)
    T = d.k.shape[0]
    assert spec_kv_append(d.k[:0], d.v[:0], d.k_cache, d.v_cache, d.args[0], d.args[1],
                          torch.zeros_like(d.args[2])) is None and T > 0


def test_append_bad_lengths_and_pages():
    b = Batch([(10, 3), (20, 4), (5, 2)], seed=6)
    k0, v0 = b.k_cache.clone(), b.v_cache.clone()
    ctx = b.args[1].clone()
    ctx[0], ctx[2] = -4, b.table.shape[1] * b.page - 1
    table = b.args[0].clone()
    table[1, 20 // b.page] = b.k_cache.shape[0]
    keep = b.args[:2]
    b.args[0], b.args[1] = table, ctx
    b.append()
    assert int(b.status) == binding.SV_FLAG_BAD_LENGTH | binding.SV_FLAG_BAD_PAGE
    assert torch.equal(b.k_cache, k0) and torch.equal(b.v_cache, v0)
    b.args[:2] = keep
    b.status.zero_()
    b.args[2] = torch.tensor([0, 40, 7, 9], dtype=torch.int32, device="cuda")  # not ascending, past T
    b.append()
    assert int(b.status) in (0, binding.SV_FLAG_BAD_LENGTH)
    bad = torch.zeros(3, 2, dtype=torch.int32, device="cuda")  # more tokens than nodes
    b.args[2] = torch.from_numpy(b.cu).cuda()
    b.k_cache.copy_(k0), b.v_cache.copy_(v0)
    b.append(tree_parents=bad)
    assert int(b.status) & binding.SV_FLAG_BAD_LENGTH
    same = (b.k_cache == k0).all(dim=(2, 3))
    stored = {(int(b.table[2, s // 16]), s % 16) for s in (5, 6)}
    assert {tuple(x) for x in (~same).nonzero().tolist()} == stored


def commit_reference(b, parents, n, last, capacity):
    k, v, lens = b.k_cache.clone(), b.v_cache.clone(), b.ctx.copy()
    for s, ctx in enumerate(b.ctx):
        if n[s] < 0:
            continue
        path = [0] if parents is None else path_to(parents[s], int(last[s]))
        if parents is not None and len(path) != n[s] + 1:
            continue
        lens[s] = ctx + 1 + n[s]
        for j, p in enumerate(path if parents is not None else []):
            src, dst = ctx + p, ctx + j
            for cache, old in ((k, b.k_cache), (v, b.v_cache)):
                cache[int(b.table[s, dst // b.page]), dst % b.page] = old[int(b.table[s, src // b.page]), src % b.page]
    return k, v, lens


@pytest.mark.parametrize("D,Hkv,layout,page", [(128, 2, "tokens", 16), (64, 1, "heads", 8), (128, 20, "halves", 24)])
def test_commit_moves_the_path(D, Hkv, layout, page):
    rng = np.random.default_rng(7)
    seqs = [(int(rng.integers(0, 50)), int(rng.integers(1, 33))) for _ in range(40)]
    b = Batch(seqs, Hkv=Hkv, D=D, page=page, layout=layout, seed=7)
    parents = np.full((40, 32), -1, np.int32)
    n, last = np.zeros(40, np.int32), np.zeros(40, np.int32)
    for s, (_, m) in enumerate(seqs):
        for i in range(1, m):
            # deep trees: long paths whose places are also nodes of the path
            parents[s, i] = max(0, i - 1 - int(rng.integers(0, 3))) if s % 2 else rng.integers(0, i)
        last[s] = rng.integers(0, m) if s % 3 else m - 1
        n[s] = len(path_to(parents[s], int(last[s]))) - 1
    k, v, lens = commit_reference(b, parents, n, last, None)
    dev = [torch.from_numpy(x).cuda() for x in (n, parents, last)]
    got = spec_kv_commit(b.k_cache, b.v_cache, b.args[0], b.args[1], dev[0], tree_parents=dev[1], last_node=dev[2],
                         status_word=b.status)
    torch.cuda.synchronize()
    assert int(b.status) == 0
    assert np.array_equal(got.cpu().numpy(), lens)
    assert torch.equal(b.k_cache, k) and torch.equal(b.v_cache, v)
    assert n.max() >= 8  # long paths are among them


def test_commit_a_chain_changes_lengths_only_and_in_place():
    b = Batch([(10, 5), (0, 1), (30, 3)], seed=8)
    k0 = b.k_cache.clone()
    n = torch.tensor([4, 0, -1], dtype=torch.int32, device="cuda")
    assert spec_kv_commit(b.k_cache, b.v_cache, b.args[0], b.args[1], n, out_lens=b.args[1], status_word=b.status) is b.args[1]
    torch.cuda.synchronize()
    assert b.args[1].tolist() == [15, 1, 30] and torch.equal(b.k_cache, k0) and int(b.status) == 0


def test_commit_refuses_what_does_not_fit():
    b = Batch([(10, 6), (10, 6), (10, 6), (10, 6)], seed=9)
    parents = np.tile(np.array([-1, 0, 1, 2, 3, 4], np.int32), (4, 1))
    parents[3, 2] = 5
    k0, v0 = b.k_cache.clone(), b.v_cache.clone()
    n = torch.tensor([6, 3, 2, 3], dtype=torch.int32, device="cuda")
    last = torch.tensor([5, 2, 9, 3], dtype=torch.int32, device="cuda")
    got = spec_kv_commit(b.k_cache, b.v_cache, b.args[0], b.args[1], n, tree_parents=torch.from_numpy(parents).cuda(),
                         last_node=last, status_word=b.status)
    torch.cuda.synchronize()
    # too many for the tree; a chain of another length; no such node; a broken chain
    assert int(b.status) == binding.SV_FLAG_BAD_LENGTH | binding.SV_FLAG_BAD_TREE
    assert got.tolist() == [10] * 4 and torch.equal(b.k_cache, k0) and torch.equal(b.v_cache, v0)
    b.status.zero_()
    room = torch.full((4,), 400, dtype=torch.int32, device="cuda")
    assert spec_kv_commit(b.k_cache, b.v_cache, b.args[0], b.args[1], room, status_word=b.status).tolist() == [10] * 4
    assert int(b.status) == binding.SV_FLAG_BAD_LENGTH


@pytest.mark.parametrize("B", [1, 40, 700])
def test_steps_back_to_back_read_the_lengths_of_the_step_before(B):
    # a graph's kernels start beside one another: append waits for the commit
    # before it, and then has to read what that wrote
    steps, page, Hkv, D = 40, 8, 1, 64
    rng = np.random.default_rng(B)
    n = rng.integers(0, 4, B).astype(np.int32)
    need = [-(-(int(x) + 1) * steps // page) + 1 for x in n]
    table = torch.from_numpy(make_table(need, sum(need) + 1, rng)).cuda()
    kc, vc = (torch.zeros(sum(need) + 1, page, Hkv, D, dtype=BF16, device="cuda") for _ in range(2))
    k, v = (torch.randn(steps, B, Hkv, D, device="cuda", generator=torch.Generator("cuda").manual_seed(B)).to(BF16) for _ in range(2))
    ctx = torch.zeros(B, dtype=torch.int32, device="cuda")
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    took, status = torch.from_numpy(n).cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")

    def run():
        for i in range(steps):
            spec_kv_append(k[i], v[i], kc, vc, table, ctx, cu, status_word=status)
            spec_kv_commit(kc, vc, table, ctx, took, out_lens=ctx, status_word=status)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    at = torch.arange(steps)[:, None] * (torch.from_numpy(n) + 1)[None]  # slot of each step's token
    pages, rows = table.cpu().gather(1, (at // page).T).T.long(), at % page
    for _ in range(5):
        kc.zero_(), vc.zero_(), ctx.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert int(status) == 0 and torch.equal(ctx.cpu(), torch.from_numpy((n + 1) * steps))
        for cache, x in ((kc, k), (vc, v)):
            got = cache.cpu()
            assert torch.equal(got[pages, rows], x.cpu())
            got[pages, rows] = 0
            assert (got == 0).all()


@pytest.mark.parametrize("seqs,cu,whole", [
    ([(10, 3), (20, 4), (5, 2)], [0, 40, 7, 9], [2]),   # ends past T, then descends
    ([(10, 3), (20, 4), (5, 2)], [-1, 3, 7, 9], [1, 2]),
    ([(10, 3), (20, 4), (5, 2)], [0, 3, 7, 10], [0, 1]),
    ([(0, 9), (20, 0), (5, 0)], [0, 9, 9, 4], [0]),     # no row lies in the one that descends
    ([(0, 9)] + [(20, 0)] * 599, [0] + [9] * 599 + [8], [0]),
])
def test_append_flags_sequences_that_are_not_rows(seqs, cu, whole):
    b = Batch(seqs, seed=10)
    want_k, want_v = b.k_cache.clone(), b.v_cache.clone()
    args = [b.args[0], b.args[1], torch.tensor(cu, dtype=torch.int32, device="cuda")]
    q_out = torch.full_like(b.q, 7.0)
    spec_kv_append(b.k, b.v, b.k_cache, b.v_cache, *args, q=b.q, q_out=q_out, status_word=b.status)
    torch.cuda.synchronize()
    assert int(b.status) == binding.SV_FLAG_BAD_LENGTH
    rows = torch.zeros(b.q.shape[0], dtype=torch.bool, device="cuda")
    for s in whole:
        for i in range(cu[s + 1] - cu[s]):
            at = int(b.table[s, (seqs[s][0] + i) // b.page]), (seqs[s][0] + i) % b.page
            want_k[at], want_v[at] = b.k[cu[s] + i], b.v[cu[s] + i]
            rows[cu[s] + i] = True
    assert torch.equal(b.k_cache, want_k) and torch.equal(b.v_cache, want_v)
    assert torch.equal(q_out[rows], b.q[rows]) and (q_out[~rows] == 7).all()


def test_append_angles_at_far_positions_of_any_frequency():
    from paged_reference import angle_far
    # x = (1, 0) gives (cos, sin); near a multiple of pi the sine shows the
    # angle's own error, 2^-24 turns at most (2 pi 2^-24 < 2^-21)
    rng = np.random.default_rng(12)
    f = np.concatenate([rng.uniform(0, 1, 24), 10.0 ** rng.uniform(0, 6, 24), -10.0 ** rng.uniform(-8, 6, 16)])
    T = 400
    pos = rng.integers(2 ** 20, 2 ** 31, T) * rng.choice([-1, 1], T)
    b = Batch([(0, T)], Hq=1, Hkv=1, dtype=FP16, seed=12)
    b.k.zero_(), b.q.zero_()
    b.k[..., :64] = b.q[..., :64] = 1.0
    q_out = b.append(q=b.q, inv_freq=torch.from_numpy(f), positions=torch.from_numpy(pos.astype(np.int32)).cuda())
    angle = np.array([[angle_far(int(p), float(w)) for w in f] for p in pos])
    slots = np.arange(T)
    k = b.k_cache[torch.from_numpy(b.table[0, slots // 16].astype(np.int64)).cuda(), torch.from_numpy(slots % 16).cuda(), 0]
    assert (np.abs(np.sin(angle)) < 2.0 ** -9).sum() > 20
    for x in (q_out[:, 0], k):
        x = x.double().cpu().numpy()
        for got, want in ((x[:, :64], np.cos(angle)), (x[:, 64:], np.sin(angle))):
            bound = 2.0 ** -11 * np.abs(want) + 1.01 * (2.0 ** -21 + 2.0 ** -22) + 2.0 ** -25
            assert (np.abs(got - want) <= bound).all(), (np.abs(got - want) / bound).max()


def test_append_of_the_most_rows_there_can_be():
    # 2^31 - 1 rows, all of them one row's memory; sequences claim the last three and two others
    T = 2 ** 31 - 1
    b = Batch([(3, 2), (0, 3)], Hkv=1, Hq=1, D=64, seed=13)
    want_k, want_v = b.k_cache.clone(), b.v_cache.clone()
    k, v = b.k[:1].expand(T, -1, -1), b.v[:1].expand(T, -1, -1)
    for s, ctx, n in ((0, 3, 2), (2, 0, 3)):
        for i in range(n):
            at = int(b.table[s // 2, (ctx + i) // 16]), (ctx + i) % 16
            want_k[at], want_v[at] = b.k[0], b.v[0]
    # a sequence between them, of all other rows, has no room: nothing is stored for it
    table = torch.cat([b.args[0][:1], b.args[0][:1], b.args[0][1:]])
    lens = torch.tensor([3, 0, 0], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 2, T - 3, T], dtype=torch.int32, device="cuda")
    spec_kv_append(k, v, b.k_cache, b.v_cache, table, lens, cu, status_word=b.status)
    torch.cuda.synchronize()
    assert int(b.status) == binding.SV_FLAG_BAD_LENGTH
    assert torch.equal(b.k_cache, want_k) and torch.equal(b.v_cache, want_v)


def test_commit_of_several_layers_that_share_their_lengths():
    layers = [Batch([(10, 6), (33, 6), (0, 6)], seed=20 + i) for i in range(3)]
    parents = np.tile(np.array([-1, 0, 0, 2, 2, 4], np.int32), (3, 1))
    n, last = np.array([3, 2, 1], np.int32), np.array([5, 3, 2], np.int32)
    dev = [torch.from_numpy(x).cuda() for x in (n, parents, last)]
    ctx = layers[0].args[1]
    want = [commit_reference(b, parents, n, last, None) for b in layers]
    for i, b in enumerate(layers):  # the last layer's call may advance the lengths in place
        spec_kv_commit(b.k_cache, b.v_cache, b.args[0], ctx, dev[0], tree_parents=dev[1], last_node=dev[2],
                       out_lens=ctx if i == 2 else torch.empty_like(ctx), status_word=b.status)
    torch.cuda.synchronize()
    for b, (k, v, lens) in zip(layers, want):
        assert int(b.status) == 0 and torch.equal(b.k_cache, k) and torch.equal(b.v_cache, v)
    assert np.array_equal(ctx.cpu().numpy(), want[0][2])
