"""Cases of the operators around a decoding step: drawing tokens and cutting
rows of logits by temperature, top-k, top-p and min-p, handing out the pages of
the cache, and paged attention whose scores are capped by a tanh or get a bias
that depends on the distance.

What a row is cut by: with the logits z of a row in descending order (equal ones
by index), w_j = exp((z_j - max z) / T), the first k remain (top-k), of these the
fewest whose w sum up to at least p times the sum of those k (top-p), and those
with w_j >= m (min-p): each keeps a beginning of the order, together the shortest
one. T = 0 keeps the first alone. A token is drawn by a given u of [0, 1): the
smallest one whose cumulative w, over what is kept and by index, is above u
times the sum.

Lengths and sizes are part of a case; values, pages and their order come from
the seed.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _logits(name, op, **kw):
    c = {"op": op, "B": 1, "rows": 1, "V": 32000, "dtype": "bf16", "cut": "mixed", "sigma": 3.0}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def _cache(name, op, **kw):
    c = {"op": op, "B": 1, "new": 1, "new_max": 1, "ctx": 0, "ctx_max": 0, "Hq": 32, "Hkv": 8, "D": 128, "page": 16,
         "dtype": "bf16", "tree": False, "cap": 0.0, "slopes": False}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one sequence's draft token, the usual cut of a chat: all latency
        _logits("sample one", "sample", dtype="fp32", cut="top-k and top-p"),
        # a serving batch whose requests each have settings of their own, some greedy
        _logits("sample batch", "sample", B=256, V=151936),
        # flat rows at a high temperature, top-p alone: the cut keeps thousands of tokens
        _logits("sample flat", "sample", B=64, V=128256, dtype="fp32", cut="top-p", sigma=1.5),
        # the target's rows of one sequence, the last token and 5 drafts
        _logits("cut one sequence", "cut", rows=6, V=32000, dtype="fp32"),
        # the target's rows as the LM head leaves them, settings by request
        _logits("cut LM head rows", "cut", B=32, rows=6, V=128256, dtype="fp32"),
        # the target's rows of a large batch with 8 drafts each: the most bytes
        _logits("cut large batch", "cut", B=256, rows=9, V=151936),
        # a step of a serving batch: 4 drafts each, some sequences need a page, some give back what they did not use
        _cache("pages of a step", "pages", B=256, new=5, new_max=5, ctx=64, ctx_max=8192),
        # long prompts arriving beside sequences that have ended
        _cache("pages of prompts", "pages", B=32, new=0, new_max=4096, ctx=0, ctx_max=2000, page=32),
        # a serving batch without drafts whose model caps its scores
        _cache("capped decode", "attention", B=128, ctx=64, ctx_max=8192, cap=30.0),
        # verification of 4 drafts by a model with a bias by distance and no rotation, 7 query heads per kv head
        _cache("biased drafts", "attention", B=33, new=5, new_max=5, ctx=33, ctx_max=4001, Hq=28, Hkv=4, D=64, page=64,
               dtype="fp16", slopes=True),
        # candidate trees of 32 nodes, capped and biased by the nodes' depths
        _cache("capped biased trees", "attention", B=64, new=32, new_max=32, ctx=200, ctx_max=2048, tree=True, cap=50.0, slopes=True),
        # a prompt's chunk over what is already cached: the largest product
        _cache("capped prompt chunk", "attention", new=2048, new_max=2048, ctx=8192, ctx_max=8192, page=64, cap=50.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("sample", "sample", "cut", "cut", "pages", "attention", "attention"))
    if op in ("sample", "cut"):
        V = _log(rng, 50, 200000)
        rows = 1 if op == "sample" and rng.random() < 0.7 else rng.randint(1, 17)
        return _logits(None, op, B=_log(rng, 1, max(1, min(400, 100_000_000 // (V * rows)))), rows=rows, V=V,
                       dtype=rng.choice(("bf16", "fp32")), sigma=rng.choice((0.5, 1.5, 3.0, 5.0)),
                       cut=rng.choice(("mixed", "mixed", "top-k", "top-p", "min-p", "top-k and top-p", "none")))
    D = rng.choice((64, 128))
    Hkv = rng.choice((1, 2, 4, 5, 8))
    G = rng.choice((1, 2, 3, 4, 7, 8)) if Hkv < 8 else rng.choice((1, 4, 5))
    kw = dict(Hq=G * Hkv, Hkv=Hkv, D=D, page=rng.choice((8, 16, 32, 48, 64, 128, 256)), dtype=rng.choice(("bf16", "fp16")))
    kw.update(rng.choice((dict(cap=30.0), dict(cap=50.0), dict(slopes=True), dict(cap=20.0, slopes=True))))
    kind = rng.choice(("decode", "verify", "tree", "prompt"))
    if kind == "prompt":
        B = _log(rng, 1, 6)
        new = _log(rng, 40, 2000 // B)
        kw.update(B=B, new=max(1, new // rng.choice((1, 2, 5))), new_max=new)
    else:
        B = _log(rng, 1, 200)
        n = {"decode": 1, "verify": rng.randint(2, 17), "tree": rng.randint(4, 32)}[kind]
        kw.update(B=B, new=n if kind == "tree" else rng.randint(1, n), new_max=n, tree=kind == "tree" and op == "attention")
    ctx_max = _log(rng, 1, max(2, min(8000 if kind == "prompt" else 20000, 200000 // kw["B"])))
    kw.update(ctx=rng.randint(0, ctx_max), ctx_max=ctx_max)
    return _cache(None, op, **kw)


def _lengths(c):
    """(context, new tokens) of each sequence, spread evenly over the case's
    ranges and paired apart."""
    B = c["B"]
    spread = lambda lo, hi, i: lo + (hi - lo) * i // max(1, B - 1)  # noqa: E731
    return [(spread(c["ctx"], c["ctx_max"], i), spread(c["new"], c["new_max"], i * 7 % B if B % 7 else i)) for i in range(B)]


def _held(i, k, n, P):
    """Pages that sequence i of the pages' cases holds before the call: for
    most what the step before needed, some more (drafts that were not kept, a
    sequence that has ended), some none yet."""
    if i % 5 == 3:
        return -(-(k + n) // P) + 1 + i % 3
    if i % 5 == 4 and n > 1:
        return 0
    return -(-k // P)


def work(c):
    if c["op"] in ("sample", "cut"):
        n = c["B"] * c["rows"]
        e = 4 if c["dtype"] == "fp32" else 2
        moved = n * c["V"] * e * (2 if c["op"] == "cut" else 1) + c["B"] * 16 + n * 12
        return {"bytes": moved, "flops": 3 * n * c["V"]}
    ln = _lengths(c)
    new, total = sum(n for _, n in ln), sum(k + n for k, n in ln)
    if c["op"] == "pages":
        before, after = [_held(i, k, n, c["page"]) for i, (k, n) in enumerate(ln)], [-(-(k + n) // c["page"]) for k, n in ln]
        change = sum(abs(x - y) for x, y in zip(before, after))
        return {"bytes": 12 * new + 4 * 2 * change + 16 * c["B"] + 8, "flops": 0}
    tables = 4 * (3 * c["B"] + sum(-(-(k + n) // c["page"]) for k, n in ln))
    # a tree's node sees the context, the root and itself at least
    pairs = sum(n * k + (2 * n - 1 if c["tree"] else n * (n + 1) // 2) for k, n in ln)
    return {"bytes": 4 * new * c["Hq"] * c["D"] + 4 * total * c["Hkv"] * c["D"] + tables, "flops": 4 * c["D"] * c["Hq"] * pairs}


class State:
    pass


def prepare(c, seed):
    dev = torch.device("cuda")
    rng, g = random.Random(seed), torch.Generator(device=dev).manual_seed(seed)
    s = State()
    s.case = c
    {"sample": _prepare_logits, "cut": _prepare_logits, "pages": _prepare_pages, "attention": _prepare_attention}[c["op"]](s, c, rng, g, dev)
    return s


def _prepare_logits(s, c, rng, g, dev):
    B, R, V = c["B"], c["rows"], c["V"]
    # many tokens that hardly matter and a few that do, the ones before a choice
    z = torch.randn(B, R, V, generator=g, device=dev, dtype=torch.float32 if c["dtype"] == "fp32" else torch.bfloat16) * c["sigma"]
    few = min(V, 24)
    at = torch.randint(0, V, (B, R, few), generator=g, device=dev)
    lift = torch.empty(B, R, few, device=dev).exponential_(generator=g) * (1.5 * c["sigma"])
    z.scatter_reduce_(2, at, (2.5 * c["sigma"] + lift).to(z.dtype), "amax")
    s.logits = z if R > 1 or c["op"] == "cut" else z.view(B, V)
    s.u = torch.rand(s.logits.shape[:-1], generator=g, device=dev)
    per = lambda values, dt: torch.tensor([rng.choice(values) for _ in range(B)], dtype=dt, device=dev)  # noqa: E731
    s.settings = {}
    if c["cut"] == "mixed":
        s.settings = {"temperature": per((0.0, 0.6, 0.8, 1.0, 1.3), torch.float32), "top_k": per((0, 0, 1, 20, 50, 200, 1000), torch.int32),
                      "top_p": per((1.0, 0.5, 0.9, 0.95, 0.99), torch.float32), "min_p": per((0.0, 0.0, 0.02, 0.1), torch.float32)}
    else:
        s.settings["temperature"] = rng.choice((0.7, 1.0, 1.2))
        if "top-k" in c["cut"]:
            s.settings["top_k"] = rng.choice((10, 50, 300))
        if "top-p" in c["cut"]:
            s.settings["top_p"] = rng.choice((0.8, 0.9, 0.95))
        if "min-p" in c["cut"]:
            s.settings["min_p"] = rng.choice((0.01, 0.05, 0.2))
    s.out = torch.empty_like(s.logits) if c["op"] == "cut" else None
    s.count = torch.empty(s.logits.shape[:-1], dtype=torch.int32, device=dev)
    s.logprobs = torch.empty(s.logits.shape[:-1], dtype=torch.float32, device=dev)


def _prepare_pages(s, c, rng, g, dev):
    P, B = c["page"], c["B"]
    ln = _lengths(c)
    rows = [(k, n, _held(i, k, n, P)) for i, (k, n) in enumerate(ln)]
    rng.shuffle(rows)
    as_int = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    starts = [0]
    for _, n, _ in rows:
        starts.append(starts[-1] + n)
    s.ctx, s.cu = as_int([r[0] for r in rows]), as_int(starts)
    wide = max(max(-(-(k + n) // P), h) for k, n, h in rows) + 1
    grant = sum(max(0, -(-(k + n) // P) - h) for k, n, h in rows)
    spare = grant + 7
    pages = sum(h for *_, h in rows) + spare
    ids = list(range(pages))
    rng.shuffle(ids)
    table, at = [[-1] * wide for _ in range(B)], spare
    for b, (_, _, h) in enumerate(rows):
        table[b][:h] = ids[at:at + h]
        at += h
    # the pool's state in one piece: the table, what each sequence holds, the stack of free pages and its height
    flat = [x for row in table for x in row] + [r[2] for r in rows] + ids[:spare] + [-1] * (pages - spare) + [spare]
    s.before = as_int(flat)
    s.pool = torch.empty_like(s.before)
    s.table, s.held, s.free, s.n_free = s.pool.split([B * wide, B, pages, 1])
    s.table = s.table.view(B, wide)
    s.slots = torch.empty(starts[-1], dtype=torch.int64, device=dev)
    s.positions = torch.empty(starts[-1], dtype=torch.int32, device=dev)


def _prepare_attention(s, c, rng, g, dev):
    dt, D, Hq, Hkv, P, B = DTYPES[c["dtype"]], c["D"], c["Hq"], c["Hkv"], c["page"], c["B"]
    ln = _lengths(c)
    rng.shuffle(ln)
    s.ctx_host, s.new_host = [k for k, _ in ln], [n for _, n in ln]
    as_int = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    starts = [0]
    for n in s.new_host:
        starts.append(starts[-1] + n)
    s.ctx, s.cu = as_int(s.ctx_host), as_int(starts)
    need = [-(-(k + n) // P) for k, n in ln]
    pages, at = sum(need) + 3, 0
    ids = list(range(pages))
    rng.shuffle(ids)
    table = [[-1] * max(need) for _ in range(B)]
    for b, n in enumerate(need):
        table[b][:n] = ids[at:at + n]
        at += n
    s.table = as_int(table)
    s.k_cache, s.v_cache = (torch.randn(pages, P, Hkv, D, generator=g, device=dev, dtype=dt) for _ in range(2))
    # scores well into the cap's bend
    s.q = torch.randn(starts[-1], Hq, D, generator=g, device=dev, dtype=dt) * (4.0 if c["cap"] else 2.0)
    s.parents = s.parents_host = None
    if c["tree"]:
        N = max(s.new_host)
        s.parents_host = [[-1] + [rng.randrange(i) for i in range(1, N)] for _ in range(B)]
        s.parents = as_int(s.parents_host)
    # 2^(-8 (h + 1) / Hq): near heads and far ones
    s.slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], device=dev) if c["slopes"] else None
    s.scale = D ** -0.5
    s.out = torch.empty_like(s.q)
    s.workspace = None
    if own:
        from speculative_decoding_verification_24_gb300 import spec_paged_attention_workspace
        s.workspace = spec_paged_attention_workspace(starts[-1], Hq, Hkv, D, device=dev)


def run(s):
    op = s.case["op"]
    if own:
        import speculative_decoding_verification_24_gb300 as sv
        if op == "sample":
            return sv.spec_sample(s.logits, s.u, **s.settings, out_logprobs=s.logprobs), s.logprobs
        if op == "cut":
            return sv.spec_truncate_logits(s.logits, **s.settings, out=s.out, out_n_kept=s.count), s.count
        if op == "pages":
            s.pool.copy_(s.before)  # a step is planned from the state that the last one left
            sv.spec_kv_pages(s.table, s.held, s.free, s.n_free, s.ctx, s.cu, s.case["page"], slots=s.slots, positions=s.positions)
            return s.pool, s.slots, s.positions
        return sv.spec_paged_attention(s.q, s.k_cache, s.v_cache, s.table, s.ctx, s.cu, scale=s.scale, tree_parents=s.parents,
                                       score_cap=s.case["cap"] or None, bias_slopes=s.slopes, out=s.out, workspace=s.workspace)
    return {"sample": _plain_sample, "cut": _plain_cut, "pages": _plain_pages, "attention": _plain_attention}[op](s)


# ------------------------------------------------------------ plain forms


def _setting(s, name, default):
    """A setting in 64 bits, one per sequence, to be met by its rows."""
    x = s.settings.get(name, default)
    if not torch.is_tensor(x):
        # a number passes through 32 bits on its way into the call
        return torch.full((s.case["B"],) + (1,) * (s.logits.dim() - 1), x, dtype=torch.float32, device=s.logits.device).double()
    return x.double().view((-1,) + (1,) * (s.logits.dim() - 1))


def _plain_kept(s):
    """Weights in 64 bits (sums next to a border decide) and which of them the
    cut keeps."""
    T, k, p, m = (_setting(s, n, d) for n, d in (("temperature", 1.0), ("top_k", 0), ("top_p", 1.0), ("min_p", 0.0)))
    V = s.logits.shape[-1]
    z, order = s.logits.sort(dim=-1, descending=True, stable=True)
    z = z.double()
    w = torch.exp((z - z[..., :1]) / torch.where(T == 0, 1.0, T))
    k = torch.where(T == 0, 1.0, torch.where(k == 0, float(V), k.clamp(max=V)))
    total = w.cumsum(-1)
    of_k = total.gather(-1, (k.long() - 1).expand(total.shape[:-1] + (1,)))
    n_p = torch.where(p >= 1, float(V), (total < p * of_k).sum(-1, keepdim=True) + 1.0)
    n_m = (w >= m).sum(-1, keepdim=True).double()
    n = torch.minimum(torch.minimum(k, n_p), n_m)
    keep = torch.arange(V, device=z.device) < n
    return torch.empty_like(w).scatter_(-1, order, w), torch.empty_like(keep).scatter_(-1, order, keep), n[..., 0].to(torch.int32)


def _plain_sample(s):
    w, keep, _ = _plain_kept(s)
    w.masked_fill_(~keep, 0.0)
    total = w.cumsum(-1)
    sum_ = total[..., -1:]
    token = (total <= s.u.double()[..., None] * sum_).sum(-1, keepdim=True).clamp(max=w.shape[-1] - 1)
    s.logprobs.copy_((w.gather(-1, token) / sum_).log()[..., 0])
    return token[..., 0].to(torch.int32), s.logprobs


def _plain_cut(s):
    _, keep, s.count = _plain_kept(s)
    s.out.copy_(s.logits.masked_fill(~keep, -math.inf))
    return s.out, s.count


def _plain_pages(s):
    P, dev = s.case["page"], s.ctx.device
    s.pool.copy_(s.before)
    n_free = s.n_free.long()
    total = (s.ctx + s.cu.diff()).long()
    need, held = (total + P - 1) // P, s.held.long()
    j = torch.arange(s.table.shape[1], device=dev)
    # what is too much goes on the stack, by sequence and place, then every
    # sequence's want is taken from its top
    back = (j >= need[:, None]) & (j < held[:, None])
    given = s.table[back]
    s.free[n_free + torch.arange(given.shape[0], device=dev)] = given
    s.table.masked_fill_(back, -1)
    top = n_free + given.shape[0]
    want = (need - held).clamp(min=0)
    before = want.cumsum(0) - want
    add = (j >= held[:, None]) & (j < need[:, None])
    at = top - 1 - (before[:, None] + j - held[:, None])
    s.table[add] = s.free[at[add]]
    s.held.copy_(need)
    s.n_free.copy_(top - want.sum())
    t = torch.arange(s.slots.shape[0], device=dev)
    b = torch.searchsorted(s.cu, t, right=True) - 1
    pos = s.ctx[b] + t - s.cu[b]
    s.slots.copy_(s.table[b, pos // P].long() * P + pos % P)
    s.positions.copy_(pos)
    return s.pool, s.slots, s.positions


def _ancestors(parents):
    """[B, N, N]: whether node j is node i or above it, by squaring the
    relation "is its parent or itself"."""
    N = parents.shape[1]
    up = torch.nn.functional.one_hot(parents.clamp(min=0).long(), N).float()
    up = torch.maximum(up, torch.eye(N, device=up.device))
    for _ in range(max(1, (N - 1).bit_length())):
        up = ((up @ up) > 0).float()
    return up > 0


def _plain_attention(s):
    c, dev = s.case, s.q.device
    B, Hkv, D, P = c["B"], c["Hkv"], c["D"], c["page"]
    G = c["Hq"] // Hkv
    n, L = max(s.new_host), max(k + m for k, m in zip(s.ctx_host, s.new_host))
    j = torch.arange(L, device=dev)
    page = s.table[:, j // P].clamp(min=0).long()
    k = s.k_cache[page, j % P].permute(0, 2, 1, 3).float()  # [B, Hkv, L, D]
    i = torch.arange(n, device=dev)
    rows = (s.cu[:-1, None] + i).clamp(max=s.q.shape[0] - 1)
    q = s.q[rows].float().view(B, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D)
    sc = ((q @ k.transpose(2, 3)) * s.scale).view(B, Hkv, n, G, L)
    del k
    if c["cap"]:
        sc = (sc / c["cap"]).tanh_() * c["cap"]
    seen = j[None, None, :] <= (s.ctx[:, None] + i)[:, :, None]  # [B, n, L]
    place, row_place = j.expand(B, L), s.ctx[:, None] + i
    if s.parents is not None:
        up = _ancestors(s.parents)
        at = j[None, :] - s.ctx[:, None]
        inside, node = (at >= 0) & (at < n), at.clamp(0, n - 1)
        tree = up.gather(2, node[:, None, :].expand(B, n, L))
        seen = torch.where(inside[:, None, :], tree, (at < 0)[:, None, :])
        depth = up.sum(-1) - 1
        place = torch.where(inside, s.ctx[:, None] + depth.gather(1, node), place)
        row_place = s.ctx[:, None] + depth
    if s.slopes is not None:
        far = (place[:, None, :] - row_place[:, :, None]).float()  # [B, n, L]
        sc = sc + s.slopes.view(1, Hkv, 1, G, 1) * far[:, None, :, None, :]
    sc = sc.masked_fill_(~seen[:, None, :, None, :], -math.inf).view(B, Hkv, n * G, L)
    sc -= sc.amax(dim=-1, keepdim=True)
    sc.exp_()
    total = sc.sum(dim=-1, keepdim=True)
    v = s.v_cache[page, j % P].permute(0, 2, 1, 3).float()
    o = (sc @ v) / total
    o = o.view(B, Hkv, n, G, D).permute(0, 2, 1, 3, 4).reshape(B, n, Hkv * G, D)
    t = torch.arange(s.q.shape[0], device=dev)
    b = torch.searchsorted(s.cu, t, right=True) - 1
    s.out.copy_(o[b, t - s.cu[b]])
    return s.out


# ------------------------------------------------- definitions in 64 bits


def _exact_row(z, T, k, p, m):
    """Mask of what one row keeps, and its weights: by the distinct values, each
    with how often it occurs."""
    values, inverse, counts = torch.unique(z, sorted=True, return_inverse=True, return_counts=True)
    w = torch.exp((values - values[-1]) / (T or 1.0))
    after = counts.flip(0).cumsum(0).flip(0)  # of this value and above
    mass = (counts * w).flip(0).cumsum(0).flip(0)
    k = 1 if T == 0 else min(k or z.numel(), z.numel())
    i = int((after >= k).nonzero()[-1])  # the value that the k-th has
    above = (int(after[i + 1]), float(mass[i + 1])) if i + 1 < len(values) else (0, 0.0)
    n = k
    if p < 1:
        bar = p * (above[1] + (k - above[0]) * float(w[i]))
        i_p = int((mass >= bar).nonzero()[-1]) if float(mass[0]) >= bar else 0
        below = (int(after[i_p + 1]), float(mass[i_p + 1])) if i_p + 1 < len(values) else (0, 0.0)
        n = min(n, below[0] + max(1, math.ceil((bar - below[1]) / float(w[i_p]))))
    enough = (w >= m).nonzero()
    n = min(n, int(after[int(enough[0])]))
    i = int((after >= n).nonzero()[-1])
    keep = inverse > i
    at = (inverse == i).nonzero()[:, 0]
    keep[at[:n - int(keep.sum())]] = True
    return keep, w[inverse], n


def _exact_logits(c, s):
    z = s.logits.reshape(-1, c["V"])
    get = lambda name, default, i: (  # noqa: E731
        s.settings[name][i // c["rows"]].item() if torch.is_tensor(s.settings.get(name)) else
        torch.tensor(s.settings.get(name, default), dtype=torch.float32).item())
    tokens, logs, counts = [], [], []
    out = z.double().clone() if c["op"] == "cut" else None
    u = s.u.reshape(-1).tolist()
    for i in range(z.shape[0]):
        keep, w, n = _exact_row(z[i].double(), get("temperature", 1.0, i), int(get("top_k", 0, i)), get("top_p", 1.0, i), get("min_p", 0.0, i))
        if out is not None:
            out[i, ~keep] = -math.inf
            counts.append(n)
            continue
        at = keep.nonzero()[:, 0]
        total = w[at].cumsum(0)
        j = min(int(torch.searchsorted(total, u[i] * total[-1], right=True)), at.numel() - 1)
        tokens.append(int(at[j]))
        logs.append(math.log(float(w[at[j]])) - math.log(float(total[-1])))
    shape = s.logits.shape[:-1]
    if out is not None:
        return out.view(s.logits.shape), torch.tensor(counts, dtype=torch.int32).view(shape)
    return torch.tensor(tokens, dtype=torch.int32).view(shape), torch.tensor(logs, dtype=torch.float64).view(shape)


def _exact_pages(c, s):
    P, wide = c["page"], s.table.shape[1]
    flat = s.before.tolist()
    B, pages = c["B"], s.free.numel()
    table = [flat[b * wide:(b + 1) * wide] for b in range(B)]
    held, free, n_free = flat[B * wide:B * wide + B], flat[B * wide + B:-1], flat[-1]
    assert len(free) == pages
    ctx, cu = s.ctx.tolist(), s.cu.tolist()
    need = [-(-(ctx[b] + cu[b + 1] - cu[b]) // P) for b in range(B)]
    for b in range(B):
        for j in range(need[b], held[b]):
            free[n_free], table[b][j] = table[b][j], -1
            n_free += 1
    slots, positions = [], []
    for b in range(B):
        for j in range(held[b], need[b]):
            n_free -= 1
            table[b][j] = free[n_free]
        for x in range(ctx[b], ctx[b] + cu[b + 1] - cu[b]):
            slots.append(table[b][x // P] * P + x % P)
            positions.append(x)
    pool = [x for row in table for x in row] + need + free + [n_free]
    return torch.tensor(pool, dtype=torch.int32), torch.tensor(slots, dtype=torch.int64), torch.tensor(positions, dtype=torch.int32)


def _node_path(parents, i):
    path = [i]
    while path[-1] > 0:
        path.append(parents[path[-1]])
    return path[::-1]


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] in ("sample", "cut"):
        return _exact_logits(c, s)
    if c["op"] == "pages":
        return _exact_pages(c, s)
    if sum(n * (x + n) for x, n in zip(s.ctx_host, s.new_host)) * c["Hq"] * c["D"] > 3e11:
        return None  # too long in 64 bits
    q, starts, G, P = s.q.double(), s.cu.tolist(), c["Hq"] // c["Hkv"], c["page"]
    out = torch.empty_like(q)
    for b in range(c["B"]):
        lo, hi, ctx = starts[b], starts[b + 1], s.ctx_host[b]
        n = hi - lo
        slot = torch.arange(ctx + n, device=q.device)
        page = s.table[b].long()[slot // P]
        kb, vb = s.k_cache[page, slot % P].double(), s.v_cache[page, slot % P].double()
        paths = [_node_path(s.parents_host[b], i) if c["tree"] else list(range(i + 1)) for i in range(n)]
        depth = torch.tensor([len(p) - 1 for p in paths], dtype=torch.float64, device=q.device)
        far = torch.cat((slot[:ctx].double() - ctx, depth)) - depth[:, None]
        mask = torch.zeros(n, ctx + n, dtype=torch.float64, device=q.device)
        mask[:, ctx:] = -math.inf
        if c["tree"]:
            for i, p in enumerate(paths):
                mask[i, [ctx + x for x in p]] = 0.0
        else:
            mask[:, ctx:].triu_(1)
        for h in range(c["Hq"]):
            sc = q[lo:hi, h] @ kb[:, h // G].T * s.scale
            if c["cap"]:
                sc = c["cap"] * torch.tanh(sc / c["cap"])
            if s.slopes is not None:
                sc = sc + s.slopes[h].double() * far
            out[lo:hi, h] = torch.softmax(sc + mask, dim=-1) @ vb[:, h // G]
    return out
