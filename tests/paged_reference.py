"""Plain references of the paged-cache operators in 64 bits, on the host and
one token at a time, with the error bounds that their tests use. Nothing here
shares code with the kernels."""
import math

import numpy as np
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
SMALLEST = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}  # half the spacing of the subnormals


def make_cache(n_pages, page, Hkv, D, dtype, g, layout="tokens"):
    """k and v [n_pages, page, Hkv, D] with N(0, 1) entries: plain, with the
    heads outside the page's entries, or as the halves of one tensor."""
    if layout == "tokens":
        k, v = (torch.randn(n_pages, page, Hkv, D, generator=g).to(dtype) for _ in range(2))
        return k.cuda(), v.cuda()
    if layout == "heads":
        k, v = (torch.randn(n_pages, Hkv, page, D, generator=g).to(dtype) for _ in range(2))
        return k.cuda().transpose(1, 2), v.cuda().transpose(1, 2)
    kv = torch.randn(n_pages, 2, page, Hkv, D, generator=g).to(dtype).cuda()
    return kv[:, 0], kv[:, 1]


def make_table(need, n_pages, rng, max_pages=None):
    """Disjoint pages in random order; unused entries hold a page number far
    out of range, which nothing may read."""
    ids = rng.permutation(n_pages)
    assert sum(need) <= n_pages
    table = np.full((len(need), max_pages or max(max(need), 1)), 1 << 30, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table


def entries(cache, table, b, slots, page):
    """[len(slots), Hkv, D] float64 of sequence b's entries."""
    slots = np.asarray(slots, np.int64)
    at = (torch.from_numpy(table[b, slots // page].astype(np.int64)), torch.from_numpy(slots % page))
    return cache.detach()[tuple(x.to(cache.device) for x in at)].cpu().double()


def path_to(parents, node):
    """The nodes from the root to `node`, or None when a parent is not an
    earlier node."""
    path = [node]
    while path[-1] > 0:
        up = int(parents[path[-1]])
        if up < 0 or up >= path[-1]:
            return None
        path.append(up)
    return path[::-1]


def visible(ctx, i, parents):
    """Slots that the chunk's token i sees."""
    if parents is None:
        return list(range(ctx + i + 1))
    path = path_to(parents, i)
    return [] if path is None else list(range(ctx)) + [ctx + p for p in path]


def attention(q, k_cache, v_cache, table, ctx, cu, page, scale, parents=None):
    """Output [T, Hq, D], lse [T, Hq] and the bounds of their errors, all
    float64. A row's weights are rounded to the cache's type (half a step of
    each, so at most that times sum w |v|), the scores are sums of D products
    in fp32 (error ds; it moves every weight by at most 2 ds relative), O sums
    in steps of 16 keys, and the output is rounded once."""
    dt = q.dtype
    T, Hq, D = q.shape
    Hkv = k_cache.shape[2]
    G = Hq // Hkv
    u = HALF_STEP[dt]
    qd = q.detach().cpu().double()
    out, bound = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, D, dtype=torch.float64)
    lse, lse_bound = torch.full((T, Hq), -math.inf, dtype=torch.float64), torch.zeros(T, Hq, dtype=torch.float64)
    for b in range(len(ctx)):
        n = int(cu[b + 1] - cu[b])
        if n == 0:
            continue
        k = entries(k_cache, table, b, range(ctx[b] + n), page)
        v = entries(v_cache, table, b, range(ctx[b] + n), page)
        for i in range(n):
            seen = visible(int(ctx[b]), i, None if parents is None else parents[b])
            if not seen:
                continue
            t = int(cu[b]) + i
            ks, vs = k[seen].transpose(0, 1), v[seen].transpose(0, 1)  # [Hkv, seen, D]
            qs = qd[t].reshape(Hkv, G, D)
            s = qs @ ks.transpose(1, 2) * scale
            ds = (qs.abs() @ ks.abs().transpose(1, 2) * scale).amax(-1) * (D + 8) * 2.0 ** -23  # [Hkv, G]
            w = torch.softmax(s, dim=-1)
            o, a = w @ vs, w @ vs.abs()
            steps = len(seen) / 16 + 16
            rel = u + 2 * ds[..., None] + steps * 2.0 ** -22
            out[t] = o.reshape(Hq, D)
            # 1.01: products of the terms
            bound[t] = 1.01 * (rel * a + u * o.abs() + u * rel * a).reshape(Hq, D) + SMALLEST[dt]
            lse[t] = torch.logsumexp(s, dim=-1).reshape(Hq)
            lse_bound[t] = (ds + (len(seen) + 64) * 2.0 ** -24).reshape(Hq) + 2.0 ** -21 * (1 + lse[t].abs())
    return out, bound, lse, lse_bound


def rotate(x, pos, inv_freq, interleaved):
    """x [H, D] float64 rotated by position pos: the value and the sum of the
    two products' magnitudes."""
    half = len(inv_freq)
    f = np.array([math.fmod(float(pos) * float(w), 2 * math.pi) if abs(pos) < 2 ** 20 else angle_far(pos, float(w))
                  for w in inv_freq])
    cos, sin = torch.from_numpy(np.cos(f)), torch.from_numpy(np.sin(f))
    a_at = torch.arange(half) * 2 if interleaved else torch.arange(half)
    b_at = a_at + 1 if interleaved else a_at + half
    out, mag = x.clone(), x.abs().clone()
    a, b = x[:, a_at], x[:, b_at]
    out[:, a_at], out[:, b_at] = a * cos - b * sin, b * cos + a * sin
    mag[:, a_at] = mag[:, b_at] = a.abs() + b.abs()
    return out, mag


def angle_far(pos, w):
    """pos * w modulo a turn with the turn's own rounding kept out: w / 2 pi as
    a 2^-80 fixed-point number."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    two_pi = Decimal("6.28318530717958647692528676655900576839433879875021164194988918")
    turns = Decimal(int(pos)) * (Decimal(w) / two_pi)
    return float((turns - turns.to_integral_value()) * two_pi)


def rotate_bound(value, mag, dtype):
    """fp32 arithmetic on angles good to 2^-24 turns (2 pi 2^-24 < 2^-21 of
    the pair's magnitude, plus 2^-22 for sine, cosine and products), then one
    rounding."""
    return HALF_STEP[dtype] * value.abs() + 1.01 * (2.0 ** -21 + 2.0 ** -22) * mag + SMALLEST[dtype]
