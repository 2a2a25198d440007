"""Cases of the paged-cache operators: appending keys and values with the
rotary rotation applied, attention of each sequence's new tokens over its
pages, and keeping a verified tree's path in the cache.

Lengths are part of a case (its work follows from them); their order over the
batch, the pages, the trees and the values come from the seed.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _case(name, op, **kw):
    c = {"op": op, "B": 1, "new": 1, "new_max": 1, "ctx": 0, "ctx_max": 0, "Hq": 32, "Hkv": 8, "D": 128, "page": 16,
         "dtype": "bf16", "tree": False, "interleaved": False, "rotary": 128, "heads_first": False}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one sequence decoding: 128 rows of one token each, all latency
        _case("append one token", "append", ctx=1000, ctx_max=1000),
        # the verify step's chunk: 64 sequences of the last token and 4 drafts
        _case("append drafts", "append", B=64, new=5, new_max=5, ctx=100, ctx_max=7000),
        # prompts of several lengths entering the cache at once, partial rotation of adjacent pairs
        _case("append prompts", "append", B=12, new=37, new_max=2900, dtype="fp16", interleaved=True, rotary=64, page=32),
        # a short dialogue, one token: the smallest call
        _case("decode one", "attention", ctx=500, ctx_max=500),
        # a serving batch without drafts, ragged contexts
        _case("decode batch", "attention", B=256, ctx=64, ctx_max=8192),
        # verification of 4 drafts over a serving batch
        _case("verify drafts", "attention", B=64, new=5, new_max=5, ctx=300, ctx_max=4096),
        # 7 query heads per kv head, 64-wide heads, cache with the heads outside the page
        _case("verify seven heads", "attention", B=33, new=1, new_max=9, ctx=33, ctx_max=3001, Hq=28, Hkv=4, D=64, page=64,
              dtype="fp16", heads_first=True),
        # candidate trees of 32 nodes
        _case("verify trees", "attention", B=64, new=32, new_max=32, ctx=200, ctx_max=2048, tree=True),
        # one long document, 8 drafts: few rows, a long cache
        _case("long context", "attention", new=9, new_max=9, ctx=131000, ctx_max=131000),
        # a prompt's chunk over what is already cached: the largest product
        _case("prompt chunk", "attention", new=4096, new_max=4096, ctx=12288, ctx_max=12288, page=64),
        # the kept paths of 64 trees, and of one
        _case("keep paths", "commit", B=64, new=32, new_max=32, ctx=200, ctx_max=2048, tree=True),
        _case("keep paths wide", "commit", B=256, new=24, new_max=24, ctx=64, ctx_max=1024, Hq=16, Hkv=16, D=128, page=32,
              dtype="fp16", tree=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "append", "attention", "attention", "attention", "attention", "commit"))
    D = rng.choice((64, 128))
    Hkv = rng.choice((1, 2, 4, 5, 8))
    G = rng.choice((1, 2, 3, 4, 7, 8)) if Hkv < 8 else rng.choice((1, 4, 5))
    kw = dict(Hq=G * Hkv, Hkv=Hkv, D=D, page=rng.choice((8, 16, 32, 48, 64, 128, 256)), dtype=rng.choice(("bf16", "fp16")),
              heads_first=rng.random() < 0.3, rotary=rng.choice((D, D, D // 2)), interleaved=rng.random() < 0.3)
    kind = rng.choice(("decode", "verify", "tree", "prompt")) if op != "commit" else "tree"
    if kind == "prompt":
        B = _log(rng, 1, 6)
        new = _log(rng, 40, 4096 // B)
        kw.update(B=B, new=max(1, new // rng.choice((1, 2, 5))), new_max=new)
    else:
        B = _log(rng, 1, 200)
        n = {"decode": 1, "verify": rng.randint(2, 17), "tree": rng.randint(4, 32)}[kind]
        kw.update(B=B, new=n if kind == "tree" else rng.randint(1, n), new_max=n, tree=kind == "tree")
    top = max(2, min(9000 if kind == "prompt" else 40000, 400000 // kw["B"]))
    ctx_max = _log(rng, 1, top)
    kw.update(ctx=rng.randint(0, ctx_max), ctx_max=ctx_max)
    return _case(None, op, **kw)


def _lengths(c):
    """(context, new tokens) of each sequence, spread evenly over the case's
    ranges and paired apart."""
    B = c["B"]
    spread = lambda lo, hi, i: lo + (hi - lo) * i // max(1, B - 1)  # noqa: E731
    return [(spread(c["ctx"], c["ctx_max"], i), spread(c["new"], c["new_max"], i * 7 % B if B % 7 else i)) for i in range(B)]


def work(c):
    e = 2
    ln = _lengths(c)
    new, total = sum(n for _, n in ln), sum(k + n for k, n in ln)
    tables = 4 * (3 * c["B"] + sum(-(-(k + n) // c["page"]) for k, n in ln))
    if c["op"] == "append":
        moved = 2 * new * (c["Hq"] + 2 * c["Hkv"]) * c["D"] * e
        return {"bytes": moved + tables, "flops": 3 * new * (c["Hq"] + c["Hkv"]) * c["rotary"]}
    if c["op"] == "commit":
        kept = sum(_kept(n, i) for i, (_, n) in enumerate(ln))
        return {"bytes": 4 * kept * c["Hkv"] * c["D"] * e + 4 * (new + 3 * c["B"]), "flops": 0}
    # a tree's node sees the context, the root and itself at least
    pairs = sum(n * k + (2 * n - 1 if c["tree"] else n * (n + 1) // 2) for k, n in ln)
    return {"bytes": 2 * new * c["Hq"] * c["D"] * e + 2 * total * c["Hkv"] * c["D"] * e + tables, "flops": 4 * c["D"] * c["Hq"] * pairs}


def _kept(n, i):
    """Accepted nodes of sequence i's tree of n nodes."""
    return min((i * 5 + 3) % 7, (n - 1) // 2)


class State:
    pass


def _inverse_frequencies(rotary):
    """10000^(-2i/rotary), on the host: what a model's configuration gives."""
    return torch.tensor([10000.0 ** (-2.0 * i / rotary) for i in range(rotary // 2)], dtype=torch.float64)


def prepare(c, seed):
    dev = torch.device("cuda")
    rng, g = random.Random(seed), torch.Generator(device=dev).manual_seed(seed)
    dt, D, Hq, Hkv, P, B = DTYPES[c["dtype"]], c["D"], c["Hq"], c["Hkv"], c["page"], c["B"]
    order = list(range(B))
    rng.shuffle(order)
    ln = _lengths(c)
    ctx, new = [ln[i][0] for i in order], [ln[i][1] for i in order]
    T, need = sum(new), [-(-(k + n) // P) for k, n in zip(ctx, new)]
    s = State()
    s.case, s.ctx_host, s.new_host = c, ctx, new
    as_int = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    s.ctx = as_int(ctx)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s.cu = as_int(starts)
    # pages in no order, as a pool hands them out after a while; a few are free
    pages = sum(need) + 3
    ids = list(range(pages))
    rng.shuffle(ids)
    table = [[-1] * max(need) for _ in range(B)]
    at = 0
    for b, n in enumerate(need):
        table[b][:n] = ids[at:at + n]
        at += n
    s.table = as_int(table)

    def cache():
        shape = (pages, Hkv, P, D) if c["heads_first"] else (pages, P, Hkv, D)
        x = torch.randn(shape, generator=g, device=dev, dtype=dt)
        return x.transpose(1, 2) if c["heads_first"] else x

    s.k_cache, s.v_cache = cache(), cache()
    # one projection's output holds queries, keys and values side by side
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=dev, dtype=dt)
    qkv[:, :Hq] *= 2.0  # attention picks some tokens over others
    s.q, s.k, s.v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    s.parents = s.kept = s.last = s.path_host = None
    if c["tree"]:
        N = max(new)
        par = [[-1] * N for _ in range(B)]
        s.path_host = []
        for b in range(B):
            for i in range(1, new[b]):
                par[b][i] = rng.randrange(i)
            # the accepted path: its nodes lie behind the places they move to
            m = _kept(new[b], order[b])
            path = sorted(rng.sample(range(m + 1, new[b]), m))
            for p, x in zip([0] + path, path):
                par[b][x] = p
            s.path_host.append([0] + path)
        s.parents = as_int(par)
        s.parents_host = par
        s.kept, s.last = as_int([len(p) - 1 for p in s.path_host]), as_int([p[-1] for p in s.path_host])
    s.inv_freq = _inverse_frequencies(c["rotary"])
    s.q_out, s.out = (torch.empty(T, Hq, D, dtype=dt, device=dev) for _ in range(2))
    s.new_ctx = torch.empty_like(s.ctx)
    s.scale = D ** -0.5
    s.workspace = None
    if own and c["op"] == "attention":
        from speculative_decoding_verification_24_gb300 import spec_paged_attention_workspace
        s.workspace = spec_paged_attention_workspace(T, Hq, Hkv, D, device=dev)
    return s


def run(s):
    op = s.case["op"]
    if own:
        import speculative_decoding_verification_24_gb300 as sv
        if op == "append":
            sv.spec_kv_append(s.k, s.v, s.k_cache, s.v_cache, s.table, s.ctx, s.cu, q=s.q, q_out=s.q_out,
                              inv_freq=s.inv_freq, interleaved=s.case["interleaved"], tree_parents=s.parents)
            return s.q_out, s.k_cache, s.v_cache
        if op == "attention":
            return sv.spec_paged_attention(s.q, s.k_cache, s.v_cache, s.table, s.ctx, s.cu, scale=s.scale,
                                           tree_parents=s.parents, out=s.out, workspace=s.workspace)
        sv.spec_kv_commit(s.k_cache, s.v_cache, s.table, s.ctx, s.kept, tree_parents=s.parents, last_node=s.last,
                          out_lens=s.new_ctx)
        return s.new_ctx, s.k_cache, s.v_cache
    return {"append": _plain_append, "attention": _plain_attention, "commit": _plain_commit}[op](s)


# ------------------------------------------------------------ plain forms


def _ancestors(parents):
    """[B, N, N]: whether node j is node i or above it, by squaring the
    relation "is its parent or itself"."""
    B, N = parents.shape
    up = torch.nn.functional.one_hot(parents.clamp(min=0).long(), N).float()
    up = torch.maximum(up, torch.eye(N, device=up.device))
    # the root's own parent entry is itself; padding nodes hang under it
    for _ in range(max(1, (N - 1).bit_length())):
        up = ((up @ up) > 0).float()
    return up > 0


def _tokens(s):
    """Sequence and place in the chunk of every packed token."""
    t = torch.arange(s.q.shape[0], device=s.q.device)
    b = torch.searchsorted(s.cu, t, right=True) - 1
    return b, t - s.cu[b]


def _rotate(x, angle, rotary, interleaved):
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x = x.float()
    r = x[..., :rotary]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = r.chunk(2, dim=-1)
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((r, x[..., rotary:]), dim=-1)


def _plain_append(s):
    c = s.case
    b, i = _tokens(s)
    slot = s.ctx[b] + i
    pos = slot
    if s.parents is not None:
        depth = _ancestors(s.parents).sum(-1) - 1
        pos = s.ctx[b] + depth[b, i]
    angle = pos.double()[:, None] * s.inv_freq.to(s.q.device, non_blocking=True)
    page, at = s.table[b, slot // c["page"]].long(), slot % c["page"]
    s.q_out.copy_(_rotate(s.q, angle, c["rotary"], c["interleaved"]))
    s.k_cache[page, at] = _rotate(s.k, angle, c["rotary"], c["interleaved"]).to(s.k.dtype)
    s.v_cache[page, at] = s.v
    return s.q_out, s.k_cache, s.v_cache


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
    sc = (q @ k.transpose(2, 3)) * s.scale
    del k
    seen = j[None, None, :] <= (s.ctx[:, None] + i)[:, :, None]  # [B, n, L]
    if s.parents is not None:
        up = _ancestors(s.parents)
        at = j[None, :] - s.ctx[:, None]
        inside = (at >= 0) & (at < n)
        tree = up.gather(2, at.clamp(0, n - 1)[:, None, :].expand(B, n, L))
        seen = torch.where(inside[:, None, :], tree, (at < 0)[:, None, :])
    seen = seen[:, None, :, None, :].expand(B, 1, n, G, L).reshape(B, 1, n * G, L)
    sc.masked_fill_(~seen, -math.inf)
    sc -= sc.amax(dim=-1, keepdim=True)
    sc.exp_()
    total = sc.sum(dim=-1, keepdim=True)
    v = s.v_cache[page, j % P].permute(0, 2, 1, 3).float()
    o = (sc @ v) / total
    o = o.view(B, Hkv, n, G, D).permute(0, 2, 1, 3, 4).reshape(B, n, Hkv * G, D)
    bt, it = _tokens(s)
    s.out.copy_(o[bt, it])
    return s.out


def _plain_commit(s):
    P, N = s.case["page"], s.parents.shape[1]
    # the path's nodes in ascending order: the nodes at or above the last one
    above = _ancestors(s.parents)[torch.arange(s.ctx.shape[0], device=s.ctx.device), s.last.long()]
    rank = above.cumsum(1) - 1
    src = s.ctx[:, None] + torch.arange(N, device=s.ctx.device)
    dst = s.ctx[:, None] + rank
    b, _ = moved = above.nonzero(as_tuple=True)
    src, dst = src[moved], dst[moved]
    for cache in (s.k_cache, s.v_cache):
        cache[s.table[b, dst // P].long(), dst % P] = cache[s.table[b, src // P].long(), src % P]
    torch.add(s.ctx, s.kept + 1, out=s.new_ctx)
    return s.new_ctx, s.k_cache, s.v_cache


# ------------------------------------------------- definitions in 64 bits


def _node_path(parents, i):
    path = [i]
    while path[-1] > 0:
        path.append(parents[path[-1]])
    return path[::-1]


def _places(s, b, slots):
    table = s.table[b].tolist()
    P = s.case["page"]
    pages = torch.tensor([table[x // P] for x in slots], device=s.q.device)
    return pages, torch.tensor([x % P for x in slots], device=s.q.device)


def exact(c, seed):
    s = prepare(c, seed)
    k, v = s.k_cache.double(), s.v_cache.double()
    q = s.q.double()
    starts = s.cu.tolist()
    if c["op"] == "commit":
        for b, path in enumerate(s.path_host):
            frm, to = _places(s, b, [s.ctx_host[b] + p for p in path]), _places(s, b, [s.ctx_host[b] + j for j in range(len(path))])
            k[to], v[to] = k[frm], v[frm]
        return torch.tensor([x + len(p) for x, p in zip(s.ctx_host, s.path_host)], dtype=torch.int32), k, v
    if c["op"] == "append":
        R = c["rotary"]
        first = torch.arange(R // 2, device=q.device) * (2 if c["interleaved"] else 1)
        second = first + (1 if c["interleaved"] else R // 2)
        f = torch.tensor([10000.0 ** (-2.0 * i / R) for i in range(R // 2)], dtype=torch.float64, device=q.device)
        kk, q_out = s.k.double(), q.clone()
        for b in range(c["B"]):
            lo, hi = starts[b], starts[b + 1]
            slots = [s.ctx_host[b] + i for i in range(hi - lo)]
            pos = slots
            if c["tree"]:
                pos = [s.ctx_host[b] + len(_node_path(s.parents_host[b], i)) - 1 for i in range(hi - lo)]
            w = torch.polar(torch.ones(1, dtype=torch.float64, device=q.device),
                            torch.tensor(pos, dtype=torch.float64, device=q.device)[:, None] * f)[:, None]
            for x in (q_out, kk):
                z = torch.complex(x[lo:hi][..., first], x[lo:hi][..., second]) * w
                x[lo:hi, :, first], x[lo:hi, :, second] = z.real, z.imag
            to = _places(s, b, slots)
            k[to], v[to] = kk[lo:hi], s.v[lo:hi].double()
        return q_out, k, v
    if sum(n * (x + n) for x, n in zip(s.ctx_host, s.new_host)) * c["Hq"] * c["D"] > 4e11:
        return None  # too long in 64 bits
    out, G = torch.empty_like(q), c["Hq"] // c["Hkv"]
    for b in range(c["B"]):
        lo, hi, ctx = starts[b], starts[b + 1], s.ctx_host[b]
        n = hi - lo
        at = _places(s, b, range(ctx + n))
        kb, vb = k[at], v[at]
        bias = torch.zeros(n, ctx + n, dtype=torch.float64, device=q.device)
        if c["tree"]:
            bias[:, ctx:] = -math.inf
            for i in range(n):
                bias[i, [ctx + p for p in _node_path(s.parents_host[b], i)]] = 0.0
        else:
            bias[:, ctx:] = torch.full((n, n), -math.inf, dtype=torch.float64, device=q.device).triu(1)
        for h in range(c["Hq"]):
            w = torch.softmax(q[lo:hi, h] @ kb[:, h // G].T * s.scale + bias, dim=-1)
            out[lo:hi, h] = w @ vb[:, h // G]
    return out
