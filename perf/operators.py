"""Cases, plain forms and 64-bit values of the token-serving operators.

The operators: `rope_append` (rotary positions applied to new queries and keys,
keys and values quantised into a paged 8-bit cache), `paged_attention` (attention
over that cache: single tokens, a few tokens, prompts; optional sliding window with
always-visible first tokens) and `sample_tokens` (temperature, top-k, top-p and
min-p from given uniform numbers).

A case is a dict of plain values.  `listed()` and `draw(rng)` give cases,
`prepare(case, seed)` the tensors a serving program holds before the call,
`run(state)` one pass: the library's kernels where `own` is true, otherwise the
plain form in elementary torch operations.  `exact(case, seed)` computes the same
outputs in 64 bits, and `work(case)` the bytes and operations of a pass.

Layout.  The cache of one layer holds pages of `page` tokens: k and v are float8
(e4m3) [pages, kv_heads, page, dim] with one float32 scale for each page and head
(value = code * scale; scales are powers of two).  The new tokens of all sequences
lie one after the other: tokens q_start[b] .. q_start[b + 1] - 1 belong to sequence
b and end at cache position kv_len[b] - 1.
"""
import math

import torch

own = False

CODE_MAX = 448.0            # largest e4m3 value
SCALE_MIN = 2.0 ** -100     # scale of a page and head whose values are all tiny or zero

ROPE_BASE = 10000.0


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one new token of one sequence in a Llama2-7B-shaped layer (32 heads of 128):
        # nothing but latency
        dict(name="append_decode_b1", op="append", batch=1, q_min=1, q_max=1, prev_min=1000, prev_max=1000,
             heads=32, kv_heads=32, dim=128, rot=128, page=64, interleaved=False, dtype="bf16"),
        # a batch that mixes decoding sequences with short prompt pieces, heads of 48
        # (the 130M stack), two thirds of each head rotated, fp32 activations
        dict(name="append_mixed_f32", op="append", batch=48, q_min=1, q_max=33, prev_min=0, prev_max=2047,
             heads=16, kv_heads=16, dim=48, rot=32, page=16, interleaved=True, dtype="f32"),
        # the prompt of a Llama2-7B-shaped layer, 4096 tokens: bound by memory
        dict(name="append_prefill", op="append", batch=1, q_min=4096, q_max=4096, prev_min=0, prev_max=0,
             heads=32, kv_heads=32, dim=128, rot=128, page=64, interleaved=False, dtype="bf16"),
        # one sequence, one new token, 4096 cached: few rows, split over the long axis
        dict(name="attn_decode_b1", op="attention", batch=1, q_min=1, q_max=1, prev_min=4095, prev_max=4095,
             heads=32, kv_heads=32, dim=128, page=64, window=0, sinks=0, dtype="bf16"),
        # a serving batch with grouped heads (8 query heads to a cached head of 64) and
        # ragged lengths from almost nothing to 4096
        dict(name="attn_decode_b128_gqa", op="attention", batch=128, q_min=1, q_max=1, prev_min=0, prev_max=4095,
             heads=32, kv_heads=4, dim=64, page=16, window=0, sinks=0, dtype="bf16"),
        # long streams of which each token sees the last 2048 and the first 4
        dict(name="attn_decode_window_sinks", op="attention", batch=8, q_min=1, q_max=1, prev_min=20000,
             prev_max=65536, heads=32, kv_heads=8, dim=128, page=32, window=2048, sinks=4, dtype="bf16"),
        # checking up to 4 proposed tokens of each sequence at once, fp32, heads of 48
        dict(name="attn_verify_f32", op="attention", batch=24, q_min=1, q_max=4, prev_min=17, prev_max=1000,
             heads=16, kv_heads=16, dim=48, page=16, window=0, sinks=0, dtype="f32"),
        # the whole prompt of a Llama2-7B-shaped layer: bound by the tensor cores
        dict(name="attn_prefill", op="attention", batch=1, q_min=4096, q_max=4096, prev_min=0, prev_max=0,
             heads=32, kv_heads=32, dim=128, page=64, window=0, sinks=0, dtype="bf16"),
        # prompt pieces of odd lengths over caches that already hold thousands of tokens
        dict(name="attn_chunks_gqa", op="attention", batch=4, q_min=257, q_max=1025, prev_min=3001, prev_max=15001,
             heads=32, kv_heads=8, dim=128, page=64, window=0, sinks=0, dtype="bf16"),
        # one row of logits over the 32000-token vocabulary: latency
        dict(name="sample_b1", op="sample", batch=1, vocab=32000, dtype="bf16"),
        # a serving batch, fp32 logits
        dict(name="sample_b64", op="sample", batch=64, vocab=32000, dtype="f32"),
        # a large batch over a large vocabulary of odd size
        dict(name="sample_b256_large", op="sample", batch=256, vocab=131071, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "prefill", "sample"])
    if op == "sample":
        c = dict(op="sample", batch=_log(rng, 1, 256), vocab=_log(rng, 100, 131072),
                 dtype=rng.choice(["bf16", "f32"]))
        if c["dtype"] == "f32":
            c["batch"] = min(c["batch"], 128)
        return c
    dim = rng.choice([48, 64, 80, 96, 128])
    page = rng.choice([16, 32, 64, 128])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 16])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "append":
        q_max = rng.choice([1, _log(rng, 2, 2048)])
        most = max(1, 4096 * 32 * 128 // (q_max * heads * dim * (2 if dtype == "f32" else 1)))
        batch = _log(rng, 1, min(256, most))
        prev = _log(rng, 1, 4096)
        return dict(op="append", batch=batch, q_min=rng.randint(1, q_max), q_max=q_max,
                    prev_min=rng.randint(0, prev), prev_max=prev, heads=heads, kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([dim, 16 * rng.randint(1, dim // 16)]), page=page,
                    interleaved=rng.random() < 0.5, dtype=dtype)
    window = rng.choice([0, 0, _log(rng, 16, 4096)])
    sinks = rng.choice([0, 4, 21]) if window else 0
    if op == "decode":
        q_max = rng.choice([1, 1, rng.randint(2, 8)])
        batch = _log(rng, 1, 128)
        prev = _log(rng, 16, 65536)
        # the cached tokens of the batch, as many bytes as the long-stream case holds at most
        prev = max(16, min(prev, 134217728 // (batch * kv_heads * dim * 2)))
    else:
        dtype = "bf16"
        q_max = _log(rng, 32, 4096)
        most = 60e9 / (4.0 * heads * dim)            # pairs of a query and a key, over all sequences
        prev = _log(rng, 1, 16384)
        while q_max * (prev + q_max) > most:
            q_max, prev = max(32, q_max * 3 // 4), prev * 3 // 4
        batch = max(1, min(8, int(most // (q_max * (prev + q_max))))) if rng.random() < 0.7 else 1
    return dict(op="attention", batch=batch, q_min=rng.randint(max(1, q_max // 4), q_max), q_max=q_max,
                prev_min=rng.randint(0, prev), prev_max=prev, heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                window=window, sinks=sinks, dtype=dtype)


def _lengths(case):
    """New and earlier tokens of each sequence: spread over their ranges, the same for
    every seed, so that the work of a case is known."""
    nq, npv = case["q_max"] - case["q_min"] + 1, case["prev_max"] - case["prev_min"] + 1
    new = [case["q_min"] + (b * 7919 + nq - 1) % nq for b in range(case["batch"])]
    prev = [case["prev_min"] + (b * 104729 + npv - 1) % npv for b in range(case["batch"])]
    return new, prev


# ------------------------------------------------------------------ inputs

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _pow2_scale(amax):
    """The smallest power of two s with amax / s <= 448, at least SCALE_MIN."""
    m, e = torch.frexp(amax)                          # amax = m * 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9).to(amax.dtype)
    s = torch.exp2(e)
    return torch.where(amax > 0, s, torch.zeros_like(s)).clamp_min(SCALE_MIN)


def _filled_cache(gen, pages, kv_heads, page, dim):
    """A cache that other requests have used before: every page holds codes."""
    x = torch.randn(pages, kv_heads, page, dim, generator=gen, device="cuda")
    # magnitudes differ from head to head and, less, from page to page
    x *= torch.exp2(torch.randn(1, kv_heads, 1, 1, generator=gen, device="cuda"))
    x *= torch.exp2(0.3 * torch.randn(pages, kv_heads, 1, 1, generator=gen, device="cuda"))
    s = _pow2_scale(x.abs().amax((2, 3)))
    return (x / s[:, :, None, None]).to(torch.float8_e4m3fn), s


def _tables(case, gen):
    """page_table, q_start, kv_len and the number of pages: the pages of a sequence lie
    anywhere in the cache."""
    new, prev = _lengths(case)
    used = [-(-(n + p) // case["page"]) for n, p in zip(new, prev)]
    pages = sum(used) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    width = max(used)
    table = torch.zeros(case["batch"], width, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    start = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda()
    length = torch.tensor([n + p for n, p in zip(new, prev)], dtype=torch.int32).cuda()
    return table, start, length, pages


def _rope_tables(positions, rot):
    inv = ROPE_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * inv
    return a.cos().float().cuda(), a.sin().float().cuda()


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = _dtype(case)
    if case["op"] == "sample":
        B, V = case["batch"], case["vocab"]
        logits = torch.randn(B, V, generator=gen, device="cuda") * 2.5
        # a few likely tokens, as a trained model has
        hot = torch.randint(0, V, (B, 24), generator=gen, device="cuda")
        logits.scatter_add_(1, hot, 10.0 * torch.rand(B, 24, generator=gen, device="cuda"))
        # some tokens are forbidden
        logits[:, torch.randint(0, V, (max(1, V // 64),), generator=gen, device="cuda")] = -math.inf
        r = torch.arange(B, device="cuda")
        return dict(
            logits=logits.to(dt), u=torch.rand(B, generator=gen, device="cuda"),
            # most requests sample, one in eight is greedy; not every request uses every filter
            temperature=torch.where(r % 8 == 7, 0.0, 0.5 + torch.rand(B, generator=gen, device="cuda")),
            top_k=torch.where(r % 3 == 1, 0, torch.randint(1, 200, (B,), generator=gen, device="cuda")).to(torch.int32),
            top_p=torch.where(r % 4 == 2, 1.0, 0.5 + 0.49 * torch.rand(B, generator=gen, device="cuda")),
            min_p=torch.where(r % 2 == 1, 0.0, 0.1 * torch.rand(B, generator=gen, device="cuda")))
    table, start, length, pages = _tables(case, gen)
    kc, ks = _filled_cache(gen, pages, case["kv_heads"], case["page"], case["dim"])
    vc, vs = _filled_cache(gen, pages, case["kv_heads"], case["page"], case["dim"])
    s = dict(k=kc, v=vc, k_scale=ks, v_scale=vs, page_table=table, q_start=start, kv_len=length)
    T, D = sum(_lengths(case)[0]), case["dim"]
    if case["op"] == "append":
        # the queries, keys and values of a token are parts of one row, as a fused
        # projection leaves them
        H, G = case["heads"], case["kv_heads"]
        x = torch.randn(T, H + 2 * G, D, generator=gen, device="cuda")
        x *= torch.exp2(torch.randn(1, H + 2 * G, 1, generator=gen, device="cuda"))
        x = x.to(dt)
        s.update(x=x, nq=x[:, :H], nk=x[:, H:H + G], nv=x[:, H + G:])
        s["cos"], s["sin"] = _rope_tables(case["prev_max"] + case["q_max"], case["rot"])
    else:
        s["q"] = (1.5 * torch.randn(T, case["heads"], D, generator=gen, device="cuda")).to(dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own and case["op"] != "sample":
        # the handles that a serving program keeps: the cache of a layer, and the batch of a
        # step, which all its layers share
        import partial_activation_sync_gb300 as caat
        s["cache"] = caat.PagedKVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["step"] = caat.PagedBatch(s["page_table"], s["q_start"], s["kv_len"], case["q_max"])
    return s


# --------------------------------------------------------------- one pass

def run(s):
    c = s["case"]
    if not own:
        return {"append": _append, "attention": _attention, "sample": _sample}[c["op"]](s, c)
    import partial_activation_sync_gb300 as caat
    if c["op"] == "append":
        q = caat.rope_append(s["nq"], s["nk"], s["nv"], s["cos"], s["sin"], s["cache"], s["step"],
                             interleaved=c["interleaved"])
        return dict(q=q, k=s["k"], v=s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    if c["op"] == "attention":
        return caat.paged_attention(s["q"], s["cache"], s["step"], window=c["window"], sinks=c["sinks"])
    return caat.sample_tokens(s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"])


def _token_places(s, T):
    """Sequence and cache position of every new token."""
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(s["q_start"][1:], t, right=True)
    return b, (s["kv_len"][b] - s["q_start"][b + 1]).long() + t


def _rotated(x, cos, sin, rot, interleaved):
    """Rotary positions on the first `rot` values of each head: pairs (2i, 2i + 1) or
    (i, i + rot / 2) turned by the angle of position and i."""
    a, rest = x[..., :rot], x[..., rot:]
    x1, x2 = (a[..., 0::2], a[..., 1::2]) if interleaved else (a[..., :rot // 2], a[..., rot // 2:])
    r1, r2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    a = torch.stack((r1, r2), -1).flatten(-2) if interleaved else torch.cat((r1, r2), -1)
    return torch.cat((a, rest), -1)


def _append(s, c):
    T, P = s["nq"].shape[0], c["page"]
    b, pos = _token_places(s, T)
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    q = _rotated(s["nq"].float(), cos, sin, c["rot"], c["interleaved"]).to(s["nq"].dtype)
    k = _rotated(s["nk"].float(), cos, sin, c["rot"], c["interleaved"])
    page, off = s["page_table"][b, pos // P].long(), pos % P
    # tokens that the page held before: those below the sequence's first new position
    first = (s["kv_len"] - s["q_start"][1:] + s["q_start"][:-1]).long()[b]
    held = torch.zeros(s["k"].shape[0], dtype=torch.long, device="cuda")
    held[page] = (first - (pos - off)).clamp(0, P)
    for x, codes, scales in ((k, s["k"], s["k_scale"]), (s["nv"].float(), s["v"], s["v_scale"])):
        _append_quantised(x, codes, scales, page, off, held)
    return dict(q=q, k=s["k"], v=s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"])


def _append_quantised(x, codes, scales, page, off, held):
    """Writes the rows x [T, heads, dim] at (page, off): a page's scale grows to hold them,
    and what the page held before is brought to the grown scale."""
    amax = torch.zeros_like(scales).scatter_reduce_(0, page[:, None].expand(-1, scales.shape[1]), x.abs().amax(-1), "amax")
    old = torch.where((held > 0)[:, None], scales, torch.zeros_like(scales))
    touched = torch.zeros(scales.shape[0], dtype=torch.bool, device="cuda")
    touched[page] = True
    new = torch.where(touched[:, None], torch.maximum(old, _pow2_scale(amax)), scales)
    at = touched.nonzero()[:, 0]
    ratio = torch.where(old[at] > 0, old[at] / new[at], torch.ones_like(new[at]))
    kept = torch.arange(codes.shape[2], device="cuda") < held[at][:, None]
    was = codes[at].float()
    codes[at] = torch.where(kept[:, None, :, None], was * ratio[:, :, None, None], was).to(codes.dtype)
    codes[page, :, off] = (x / new[page][..., None]).clamp(-CODE_MAX, CODE_MAX).to(codes.dtype)
    scales.copy_(new)


def _visible(case, qpos, kpos):
    """Whether a query at qpos sees the key at kpos."""
    see = kpos <= qpos
    if case["window"]:
        see = see & ((kpos > qpos - case["window"]) | (kpos < case["sinks"]))
    return see


def _attention(s, c):
    T, H, D = s["q"].shape
    G, P, B = c["kv_heads"], c["page"], c["batch"]
    table = s["page_table"].long()
    L = table.shape[1] * P

    def gathered(codes, scales):                       # [B, G, L, D]
        return (codes[table].float() * scales[table][..., None, None]).transpose(1, 2).reshape(B, G, L, D)

    # the new tokens of each sequence side by side: [B, q_max]
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    i = torch.arange(c["q_max"], device="cuda")
    inside = i < n[:, None]
    at = (s["q_start"][:-1].long()[:, None] + i).clamp_max(T - 1)
    qpos = (s["kv_len"].long() - n)[:, None] + i
    kpos = torch.arange(L, device="cuda")
    see = _visible(c, qpos[:, :, None], kpos) & inside[:, :, None] & (kpos < s["kv_len"].long()[:, None, None])
    see = see[:, None, None]                           # [B, 1, 1, q_max, L]
    q = s["q"][at].float().reshape(B, -1, G, H // G, D).permute(0, 2, 3, 1, 4)
    scores = (q.reshape(B, G, -1, D) @ gathered(s["k"], s["k_scale"]).transpose(2, 3)) * (D ** -0.5)
    scores = scores.reshape(B, G, H // G, -1, L).masked_fill_(~see, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(B, G, -1, L) @ gathered(s["v"], s["v_scale"])).reshape(B, G, H // G, -1, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    o = o.permute(0, 3, 1, 2, 4).reshape(B, -1, H, D)
    b, _ = _token_places(s, T)
    return o[b, torch.arange(T, device="cuda") - s["q_start"][b].long()].to(s["q"].dtype)


def _sample(s, c):
    z = s["logits"].float()
    top = z.amax(-1, keepdim=True)
    greedy = s["temperature"] <= 0
    t = torch.where(greedy, torch.ones_like(s["temperature"]), s["temperature"])[:, None]
    order, index = torch.sort(z, dim=-1, descending=True, stable=True)       # ties: lowest index first
    rank = torch.arange(c["vocab"], device="cuda")
    w = ((order - top) / t).exp()
    k = torch.where(s["top_k"] > 0, s["top_k"], c["vocab"])[:, None]
    w = torch.where(rank < k, w, torch.zeros_like(w))
    # the answer is a whole number: the running sums are in 64 bits, so that it does not turn
    # on the rounding of 131072 additions
    before = w.cumsum(-1, dtype=torch.float64) - w
    keep = (before < s["top_p"][:, None] * w.sum(-1, keepdim=True, dtype=torch.float64)) | (s["top_p"][:, None] >= 1)
    keep = (keep & (w >= s["min_p"][:, None])) | (rank == 0)
    w = torch.zeros_like(w).scatter_(1, index, torch.where(keep, w, torch.zeros_like(w)))
    running = w.cumsum(-1, dtype=torch.float64)
    token = (running <= s["u"][:, None] * running[:, -1:]).sum(-1).clamp_max(c["vocab"] - 1)
    token = torch.where(greedy, index[:, 0], token)
    logprob = (z.gather(1, token[:, None]) - top)[:, 0] - (z - top).exp().sum(-1).log()
    return token.to(torch.int32), logprob


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "sample":
        # the tokens are whole numbers; the log probability belongs to the token drawn
        s["case"] = case
        token = _sample(s, case)[0].long()
        z = s["logits"].double()
        return None, torch.log_softmax(z, -1).gather(1, token[:, None])[:, 0]
    return _exact_append(case, s) if case["op"] == "append" else _exact_attention(case, s)


def _exact_code(x):
    """x (64 bits) rounded to the nearest e4m3 value, ties to even, at most 448."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp_min(-6).double() - 3)
    return (torch.round(x / step) * step).clamp(-CODE_MAX, CODE_MAX)


def _exact_append(case, s):
    new, prev = _lengths(case)
    P, rot = case["page"], case["rot"]
    out = {n: s[n].double() for n in ("k", "v", "k_scale", "v_scale")}
    qs = []
    half = torch.arange(rot, device="cuda")
    if case["interleaved"]:
        first, partner, sign = half // 2, half ^ 1, torch.where(half % 2 == 0, -1.0, 1.0).double()
    else:
        first, partner = half % (rot // 2), (half + rot // 2) % rot
        sign = torch.where(half < rot // 2, -1.0, 1.0).double()
    at = 0
    for b, (n, p) in enumerate(zip(new, prev)):
        cos, sin = s["cos"][p:p + n].double()[:, None, first], s["sin"][p:p + n].double()[:, None, first]

        def turned(x):
            y = x.double().clone()
            y[..., :rot] = y[..., :rot] * cos + sign * y[..., partner] * sin
            return y

        qs.append(turned(s["nq"][at:at + n]))
        rows = {"k": turned(s["nk"][at:at + n]), "v": s["nv"][at:at + n].double()}
        for j in range(p // P, (p + n - 1) // P + 1):
            lo, hi = max(p, j * P), min(p + n, (j + 1) * P)
            page, held = int(s["page_table"][b, j]), lo - j * P
            for name, x in rows.items():
                piece = x[lo - p:hi - p].transpose(0, 1)                       # [heads, tokens, dim]
                big = piece.abs().amax((1, 2))
                need = torch.exp2(torch.ceil(torch.log2(big / CODE_MAX)))
                # a logarithm rounded across a whole number is one power of two off
                need = torch.where(need * CODE_MAX / 2 >= big, need / 2, need)
                need = torch.where(need * CODE_MAX < big, need * 2, need).clamp_min(SCALE_MIN)
                old = out[name + "_scale"][page] if held else torch.zeros_like(need)
                scale = torch.maximum(old, need)
                if held:
                    was = out[name][page, :, :held]
                    out[name][page, :, :held] = _exact_code(was * (old / scale)[:, None, None])
                out[name][page, :, held:held + hi - lo] = _exact_code(piece / scale[:, None, None])
                out[name + "_scale"][page] = scale
        at += n
    return dict(out, q=torch.cat(qs))


def _exact_attention(case, s):
    new, prev = _lengths(case)
    if sum(n * (n + p) for n, p in zip(new, prev)) * case["heads"] * case["dim"] > 4e12:
        return None
    G, P = case["kv_heads"], case["page"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, p) in enumerate(zip(new, prev)):
        L = n + p
        pages = s["page_table"][b, :-(-L // P)].long()
        see = _visible(case, torch.arange(p, L, device="cuda")[:, None], torch.arange(L, device="cuda"))
        for g in range(G):
            k = (s["k"][pages, g].double() * s["k_scale"][pages, g, None, None].double()).flatten(0, 1)[:L]
            v = (s["v"][pages, g].double() * s["v_scale"][pages, g, None, None].double()).flatten(0, 1)[:L]
            for h in range(g * (case["heads"] // G), (g + 1) * (case["heads"] // G)):
                a = (s["q"][at:at + n, h].double() @ k.T) / math.sqrt(case["dim"])
                out[at:at + n, h] = torch.softmax(a.masked_fill(~see, -math.inf), -1) @ v
        at += n
    return out


# ------------------------------------------------------------------- work

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    B = case["batch"]
    if case["op"] == "sample":
        # logits once; a weight and its sum for every token, four numbers in and two out a row
        return dict(bytes=B * case["vocab"] * es + B * 28, flops=B * case["vocab"] * 4)
    new, prev = _lengths(case)
    T, H, G, D, P = sum(new), case["heads"], case["kv_heads"], case["dim"], case["page"]
    pages = [(n + p - 1) // P - p // P + 1 for n, p in zip(new, prev)]
    if case["op"] == "append":
        # queries in and out, keys and values in, codes out; scales of the touched pages;
        # one row of the angle tables for every token
        b = T * D * (2 * H * es + 2 * G * es + 2 * G) + sum(pages) * G * 2 * 8 + T * case["rot"] * 4
        return dict(bytes=b, flops=T * ((H + G) * case["rot"] * 3 + 2 * G * D * 2))
    pairs, keys = 0, 0
    w, k = case["window"], case["sinks"]
    for n, p in zip(new, prev):
        if w:
            for i in range(p, p + n):
                pairs += min(i + 1, w) + min(k, max(0, i + 1 - w))
            lo = max(0, p + 1 - w)                    # first key of the first query's window
            keys += p + n - lo + min(k, lo)
        else:
            pairs += n * p + n * (n + 1) // 2
            keys += n + p
    b = 2 * T * H * D * es + 2 * keys * G * D + 2 * 4 * G * -(-keys // P) + 4 * -(-keys // P)
    return dict(bytes=b, flops=4 * pairs * H * D)
