"""spec_kv_pages against a loop over the sequences, and with the paged cache's
other operators."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

BAD_LENGTH, BAD_PAGE, NO_PAGES = 64, 512, 2048


def api():
    import speculative_decoding_verification_24_gb300 as sv
    return sv


class Pool:
    """The pool's state on the host, and the definition."""

    def __init__(self, table, held, free, n_free, n_pages):
        self.table, self.held, self.n_free, self.n_pages = [r[:] for r in table], held[:], n_free, n_pages
        self.free = free[:] + [-7] * (n_pages - len(free))

    def step(self, ctx, cu, P, T):
        B, wide, flags = len(ctx), len(self.table[0]), 0
        rows_ok = [0 <= cu[b] <= cu[b + 1] <= T for b in range(B)]
        n = [cu[b + 1] - cu[b] for b in range(B)]
        ok = [rows_ok[b] and ctx[b] >= 0 and 0 <= self.held[b] <= wide and ctx[b] + n[b] <= wide * P for b in range(B)]
        need = [-(-(ctx[b] + n[b]) // P) if ok[b] else self.held[b] for b in range(B)]
        back = sum(max(0, self.held[b] - need[b]) for b in range(B) if ok[b])
        slots, positions = [-1] * T, [-1] * T
        if not all(rows_ok) or not 0 <= self.n_free <= self.n_pages or self.n_free + back > self.n_pages:
            return slots, positions, BAD_LENGTH
        flags |= 0 if all(ok) else BAD_LENGTH
        valid = lambda p: 0 <= p < self.n_pages  # noqa: E731
        for b in range(B):
            if ok[b]:
                for j in range(need[b], self.held[b]):
                    flags |= 0 if valid(self.table[b][j]) else BAD_PAGE
                    self.free[self.n_free], self.table[b][j] = self.table[b][j], -1
                    self.n_free += 1
        short = False
        for b in range(B):
            want = max(0, need[b] - self.held[b])
            if want and (short or want > self.n_free):
                short, flags = True, flags | NO_PAGES
            elif want:
                for j in range(self.held[b], need[b]):
                    self.n_free -= 1
                    self.table[b][j] = self.free[self.n_free]
                    flags |= 0 if valid(self.table[b][j]) else BAD_PAGE
                self.held[b] = need[b]
            else:
                self.held[b] = need[b]
            if not ok[b]:
                continue
            for i in range(n[b]):
                x = ctx[b] + i
                positions[cu[b] + i] = x
                if x // P < self.held[b]:
                    page = self.table[b][x // P]
                    if valid(page):
                        slots[cu[b] + i] = page * P + x % P
                    else:
                        flags |= BAD_PAGE
        return slots, positions, flags

    def device(self, extra=0):
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        table = i32([r + [9] * extra for r in self.table])[:, :len(self.table[0])]
        return [table, i32(self.held), i32(self.free), i32([self.n_free])]


def compare(pool, ctx, cu, P, T, extra=0):
    sv = api()
    dev = pool.device(extra)
    slots, positions = torch.full((T,), 5, dtype=torch.int64, device="cuda"), torch.full((T,), 5, dtype=torch.int32, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    sv.spec_kv_pages(*dev, i32(ctx), i32(cu), P, slots=slots, positions=positions, status_word=flags)
    want = pool.step(ctx, cu, P, T)
    assert slots.tolist() == want[0] and positions.tolist() == want[1]
    assert flags.item() == want[2]
    assert dev[0].tolist() == pool.table and dev[1].tolist() == pool.held and dev[3].item() == pool.n_free
    assert dev[2].tolist() == pool.free
    if extra:
        assert (dev[0]._base[:, len(pool.table[0]):] == 9).all()
    return want[2]


def make(rng, B, wide, n_pages, held, spare):
    ids = list(range(n_pages))
    rng.shuffle(ids)
    table, at = [[-1] * wide for _ in range(B)], spare
    for b in range(B):
        table[b][:held[b]] = ids[at:at + held[b]]
        at += held[b]
    assert at <= n_pages
    return Pool(table, held, ids[:spare], spare, n_pages)


def starts(n):
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    return cu


@pytest.mark.parametrize("B,P,longest,most_new", ((1, 16, 40, 1), (1, 8, 5000, 3000), (3, 64, 300, 7), (33, 16, 500, 9), (512, 16, 200, 5),
                                                  (513, 24, 100, 33), (2000, 8, 60, 2), (8192, 16, 40, 3)))
def test_steps(B, P, longest, most_new):
    """Three steps of growing, shrinking, ending and starting sequences."""
    rng = random.Random(B * 1000 + P)
    wide = -(-(longest + most_new) // P) + 2
    held = [rng.choice((0, rng.randint(0, wide))) for _ in range(B)]
    spare = B * wide - sum(held) + 3
    pool = make(rng, B, wide, sum(held) + spare, held, spare)
    for _ in range(3):
        ctx = [rng.choice((0, rng.randint(0, longest), max(0, min(longest, h * P - rng.randint(0, P))))) for h in pool.held]
        n = [rng.choice((0, 1, rng.randint(0, most_new))) for _ in range(B)]
        T = sum(n) + rng.choice((0, 5))
        assert compare(pool, ctx, starts(n), P, T, extra=rng.choice((0, 3))) == 0


def test_rows_before_the_first_and_behind_the_last_sequence():
    rng = random.Random(5)
    pool = make(rng, 3, 4, 20, [1, 0, 2], 17)
    assert compare(pool, [3, 0, 30], [4, 9, 9, 12], 16, 40) == 0


def test_too_few_pages():
    """The first that asks for too much gets none, nor do later ones; those that
    ask for nothing go on."""
    for spare in range(9):
        rng = random.Random(spare)
        pool = make(rng, 5, 8, 10 + spare, [1, 2, 4, 0, 1], spare)
        # wants 2, 3, gives 1 back, wants 1, nothing
        flags = compare(pool, [16, 40, 40, 0, 10], starts([20, 33, 3, 2, 6]), 16, 64)
        assert flags == (0 if spare >= 5 else NO_PAGES)


def test_what_is_left_out():
    rng = random.Random(2)
    assert compare(make(rng, 4, 4, 30, [1, 1, 2, 0], 9), [-1, 60, 70, 0], starts([1, 1, 5, 3]), 16, 12) == BAD_LENGTH
    pool = make(rng, 3, 4, 30, [1, 1, 2], 9)
    pool.held[1] = 5
    assert compare(pool, [3, 4, 5], starts([1, 1, 1]), 16, 3) == BAD_LENGTH
    for cu in ([0, 5, 3, 6], [-1, 2, 3, 4], [0, 2, 4, 99]):
        assert compare(make(rng, 3, 4, 30, [1, 1, 2], 9), [3, 4, 5], cu, 16, 12) == BAD_LENGTH
    for n_free in (-1, 31):
        pool = make(rng, 3, 4, 30, [1, 1, 2], 9)
        pool.n_free = n_free
        assert compare(pool, [3, 4, 5], starts([1, 1, 1]), 16, 3) == BAD_LENGTH
    pool = make(rng, 3, 4, 30, [1, 4, 2], 9)
    pool.n_free = 29  # with what comes back there are more than 30
    assert compare(pool, [3, 4, 5], starts([1, 1, 1]), 16, 3) == BAD_LENGTH


def test_bad_pages_move_as_they_are():
    rng = random.Random(3)
    pool = make(rng, 4, 6, 30, [2, 4, 1, 0], 5)
    pool.table[0][1], pool.table[1][3], pool.free[4] = 30, -5, 1 << 30
    assert compare(pool, [20, 20, 10, 0], starts([3, 2, 30, 40]), 16, 75) == BAD_PAGE


def test_without_rows_and_one_of_them():
    sv = api()
    rng = random.Random(4)
    for keep in ((), ("slots",), ("positions",)):
        pool = make(rng, 3, 4, 20, [1, 0, 4], 15)
        dev = pool.device()
        ctx, cu = [10, 0, 20], starts([10, 5, 0])
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        out = {"slots": torch.empty(15, dtype=torch.int64, device="cuda"), "positions": torch.empty(15, dtype=torch.int32, device="cuda")}
        sv.spec_kv_pages(*dev, i32(ctx), i32(cu), 16, **{k: out[k] for k in keep})
        slots, positions, _ = pool.step(ctx, cu, 16, 15)
        assert dev[0].tolist() == pool.table and dev[3].item() == pool.n_free
        if "slots" in keep:
            assert out["slots"].tolist() == slots
        if "positions" in keep:
            assert out["positions"].tolist() == positions


def test_slots_are_where_the_append_writes():
    """A few steps in one graph: pages, append, attention's lengths; what the
    append writes lies at the slots, and no page has two owners."""
    sv = api()
    B, P, wide, Hkv, D, n = 6, 16, 12, 2, 64, 5
    n_pages = B * wide
    rng = random.Random(7)
    pool = make(rng, B, wide, n_pages, [0] * B, n_pages)
    table, held, free, n_free = pool.device()
    kc, vc = (torch.zeros(n_pages, P, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ctx = torch.tensor([0, 3, 16, 30, 11, 47], dtype=torch.int32, device="cuda")
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * n
    k, v = (torch.randn(B * n, Hkv, D, device="cuda").to(torch.bfloat16) for _ in range(2))
    slots, kept = torch.empty(B * n, dtype=torch.int64, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step():
        sv.spec_kv_pages(table, held, free, n_free, ctx, cu, P, slots=slots, status_word=flags)
        sv.spec_kv_append(k, v, kc, vc, table, ctx, cu, status_word=flags)
        sv.spec_kv_commit(kc, vc, table, ctx, kept, out_lens=ctx, status_word=flags)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(20):
        kept.fill_(i % n)
        k.normal_()
        graph.replay()
        assert torch.equal(kc.view(-1, Hkv, D)[slots], k)
        owned = [table[b, :held[b]].tolist() for b in range(B)]
        pages = sum(owned, []) + free[:n_free.item()].tolist()
        assert sorted(pages) == list(range(n_pages))
        if i == 9:
            ctx.zero_()
    assert flags.item() == 0
