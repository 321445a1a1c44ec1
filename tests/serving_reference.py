"""Plain forms of the serving operators on the CPU, written from their formulas:
attention and sampling in 64 bits, the append in the separately rounded fp32 steps
its definition fixes (so its results are compared bit for bit)."""
import math

import numpy as np
import torch


def make_tables(lens_new, lens_kv, page, width=None, spare=2, seed=0):
    """page_table [B, width], q_start, kv_len as int32 CPU tensors, and the page count:
    the pages of each sequence scattered over the cache."""
    used = [-(-n // page) for n in lens_kv]
    total = sum(used) + spare
    order = np.random.default_rng(seed).permutation(total).astype(np.int32)
    width = max(max(used), 1) if width is None else width
    table = np.zeros((len(lens_kv), width), np.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    start = np.concatenate([[0], np.cumsum(lens_new)]).astype(np.int32)
    return (torch.from_numpy(table), torch.from_numpy(start), torch.tensor(lens_kv, dtype=torch.int32), total)


def cached(codes, scale, table, b, h, n, page):
    """The first n cached rows of sequence b and head h, in 64 bits."""
    out = torch.zeros(n, codes.shape[-1], dtype=torch.float64)
    for j in range(-(-n // page)):
        pg = int(table[b, j])
        m = min(page, n - j * page)
        out[j * page:j * page + m] = codes[pg, h, :m].double() * float(scale[pg, h])
    return out


def attention(q, k, v, ks, vs, table, start, kv_len, page, scale, window=0, sinks=0):
    """(out, spread) in 64 bits; spread = sum_j p_j |v_j|, the scale of the rounding of
    the weights.  All arguments on the CPU."""
    T, H, D = q.shape
    G = k.shape[1]
    g = H // G
    out = torch.zeros(T, H, D, dtype=torch.float64)
    spread = torch.zeros_like(out)
    for b in range(len(kv_len)):
        t0, t1, L = int(start[b]), int(start[b + 1]), int(kv_len[b])
        for h in range(G):
            kk, vv = cached(k, ks, table, b, h, L, page), cached(v, vs, table, b, h, L, page)
            for t in range(t0, t1):
                p = L - (t1 - t0) + t - t0
                j = torch.arange(L)
                see = (j <= p) & ((j > p - window) | (j < sinks) if window else torch.ones(L, dtype=torch.bool))
                if not see.any():
                    continue
                for i in range(h * g, (h + 1) * g):
                    s = kk[see] @ q[t, i].double() * scale
                    w = torch.softmax(s, 0)
                    out[t, i] = (w[:, None] * vv[see]).sum(0)
                    spread[t, i] = (w[:, None] * vv[see].abs()).sum(0)
    return out, spread


def pow2_scale(m):
    """Least power of two s with m / s <= 448, not below 2^-100."""
    if not m > 0:
        return 2.0 ** -100
    s = 2.0 ** (math.floor(math.log2(m)) - 12)
    while m / s > 448:
        s *= 2
    return max(s, 2.0 ** -100)


def rotated(x, cos, sin, rot, interleaved):
    """fp32 rows [..., dim] at one position: each product and sum rounded once."""
    y = x.clone()
    if rot == 0:
        return y
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = ra, rb
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = ra, rb
    return y


def append(q, k, v, cos, sin, rot, interleaved, kc, vc, ks, vs, table, start, kv_len, page):
    """Returns the rotated queries (fp32) and changes the CPU cache in place."""
    qo = torch.zeros(q.shape, dtype=torch.float32)
    for b in range(len(kv_len)):
        t0, t1, L = int(start[b]), int(start[b + 1]), int(kv_len[b])
        first = L - (t1 - t0)
        lo = max(first, 0)
        at = lambda x, p: x[p] if rot else None  # noqa: E731
        for p in range(lo, L):
            qo[t0 + p - first] = rotated(q[t0 + p - first].float(), at(cos, p), at(sin, p), rot, interleaved)
        for j in range(lo // page, -(-L // page)):
            a, e = max(lo, j * page), min(L, (j + 1) * page)
            if a >= e:
                continue
            pg, held = int(table[b, j]), a - j * page
            for codes, scales, src, turn in ((kc, ks, k, True), (vc, vs, v, False)):
                rows = torch.stack([rotated(src[t0 + p - first].float(), at(cos, p), at(sin, p), rot, interleaved)
                                    if turn else src[t0 + p - first].float() for p in range(a, e)], 1)
                for h in range(rows.shape[0]):
                    x = rows[h]
                    fin = x[torch.isfinite(x)].abs()
                    need = pow2_scale(float(fin.max()) if fin.numel() else 0.0)
                    old = float(scales[pg, h]) if held else 0.0
                    new = max(old, need)
                    if held and new > old:
                        codes[pg, h, :held] = (codes[pg, h, :held].float() * (old / new)).to(codes.dtype)
                    codes[pg, h, held:held + e - a] = (x / new).clamp(-448, 448).to(codes.dtype)
                    scales[pg, h] = new
    return qo


def sample(z, u, temperature, top_k, top_p, min_p):
    """One row, 64 bits: (token, log softmax(z)[token])."""
    z = z.astype(np.float64).copy()
    z[np.isnan(z)] = -np.inf
    V = z.size
    order = np.lexsort((np.arange(V), -z))
    top = z[order[0]]
    if top == -np.inf:
        return -1, -math.inf
    with np.errstate(invalid="ignore", over="ignore"):
        gap = np.where(z == top, 0.0, z - top)
        lse = math.log(np.exp(gap).sum())
        if temperature <= 0:
            return int(order[0]), -lse
        w = np.where(gap == -np.inf, 0.0, np.exp(gap / temperature))[order]
    if 0 < top_k < V:
        w[top_k:] = 0
    before = np.cumsum(w) - w
    keep = np.ones(V, bool) if top_p >= 1 else before < top_p * w.sum()
    keep &= w >= min_p
    keep[0] = True
    kept = np.zeros(V)
    kept[order] = np.where(keep, w, 0)
    run = np.cumsum(kept)
    hit = np.nonzero((run > u * run[-1]) & (kept > 0))[0]
    token = int(hit[0]) if hit.size else int(np.nonzero(kept)[0][-1])
    return token, float(gap[token] - lse)
