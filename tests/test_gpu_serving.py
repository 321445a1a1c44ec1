"""Rotary append to the paged 8-bit cache, attention over it and sampling, on the GPU
against plain forms on the CPU (tests/serving_reference.py)."""
import math

import numpy as np
import pytest
import torch

import partial_activation_sync_gb300 as caat
import serving_reference as ref

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _cache(seed, pages, heads, page, dim, spread=1.0):
    """CPU codes and power-of-two scales that differ from page to page."""
    g = _gen(seed)
    codes = [(torch.randn(pages, heads, page, dim, generator=g) * 90).clamp(-448, 448).to(F8) for _ in range(2)]
    scales = [torch.exp2(torch.round(spread * torch.randn(pages, heads, generator=g)) - 6) for _ in range(2)]
    return codes[0], codes[1], scales[0], scales[1]


def _handles(k, v, ks, vs, table, start, length, q_max):
    cache = caat.PagedKVCache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda())
    return cache, caat.PagedBatch(table.cuda(), start.cuda(), length.cuda(), q_max)


def _same_bits(a, b):
    a, b = a.cpu(), b.cpu()
    if a.dtype == F8:
        a, b = a.float(), b.float()
    return bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


# --------------------------------------------------------------- attention

# Bounds of an output element, with A = sum_j p_j |v_j| in 64 bits.
#   bf16: the output's rounding is 2^-9 of it.  The weights are f16: 2^-12 of each, at
#   most 2^-12 A in all; 2^-10 A leaves a factor 4 for the scores and exponentials, whose
#   errors (fp32, scores below 32) stay under 2^-15 A.
#   fp32: operands in two f16 halves (2^-22 of each) and fp32 sums.  A score below 32 is
#   off by at most about 32 * 2^-22 = 2^-17, and so is a weight, relatively; 2^-15 A
#   leaves a factor 4.
BOUND = {"bf16": (2.0 ** -8, 2.0 ** -10), "f32": (2.0 ** -22, 2.0 ** -15)}


def _check_attention(got, want, spread, dtype):
    got = got.double().cpu()
    rel, tau = BOUND[dtype]
    bad = ~((got - want).abs() <= rel * want.abs() + tau * spread)
    bad &= ~(torch.isnan(got) & torch.isnan(want))
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist())


def _attention(new, kv, heads, kv_heads, dim, page, dtype, window=0, sinks=0, seed=0, spread=1.0, edit=None, q_scale=1.0):
    table, start, length, pages = ref.make_tables(new, kv, page, seed=seed)
    k, v, ks, vs = _cache(seed + 1, pages, kv_heads, page, dim, spread)
    q = (torch.randn(sum(new), heads, dim, generator=_gen(seed + 2)) * q_scale).to(DT[dtype])
    if edit is not None:
        edit(q, k, v, ks, vs, table)
    scale = 0.4 / math.sqrt(dim)
    want, width = ref.attention(q, k, v, ks, vs, table, start, length, page, scale, window, sinks)
    cache, batch = _handles(k, v, ks, vs, table, start, length, max(new))
    got = caat.paged_attention(q.cuda(), cache, batch, softmax_scale=scale, window=window, sinks=sinks)
    assert caat.device_status() == 0
    _check_attention(got, want, width, dtype)
    return got, want


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [16, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("page", [16, 64])
def test_attention_one_token(dtype, dim, page):
    _attention([1, 1, 1, 1, 1], [1, 15, 16, 77, 300], 4, 2, dim, page, dtype, seed=dim)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (6, 2), (8, 1), (12, 4), (9, 1), (16, 1), (24, 1), (64, 2)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_groups(heads, kv_heads, dtype):
    _attention([1, 1], [33, 128], heads, kv_heads, 64, 32, dtype, seed=heads)


@pytest.mark.parametrize("new,kv", [([3], [3]), ([5, 1, 7, 2], [5, 40, 131, 2]), ([17], [200]), ([70], [133]),
                                    ([1, 40, 0, 9], [12, 40, 50, 300]), ([129, 200], [129, 391])])
@pytest.mark.parametrize("heads,kv_heads,dim,page", [(2, 2, 128, 64), (6, 2, 64, 16), (8, 1, 48, 128), (5, 1, 96, 32)])
def test_attention_several_tokens(new, kv, heads, kv_heads, dim, page):
    _attention(new, kv, heads, kv_heads, dim, page, "bf16", seed=sum(new))


def test_attention_several_tokens_f32():
    _attention([5, 1, 19], [5, 40, 131], 6, 2, 48, 16, "f32", seed=3)


@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (33, 1), (100, 21), (7, 64), (1000, 4)])
@pytest.mark.parametrize("new", [[1, 1, 1], [4, 2, 9], [150, 40, 33]])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_window_and_first_tokens(window, sinks, new, dtype):
    if dtype == "f32" and max(new) > 9:
        new = [20, 5, 1]
    _attention(new, [n + p for n, p in zip(new, (250, 17, 0))], 4, 2, 64, 16, dtype, window, sinks, seed=window)


def test_attention_long_split_over_blocks():
    # one sequence over many blocks of a cluster, with an odd tail
    _attention([1], [5003], 4, 1, 128, 64, "bf16", seed=5)
    _attention([1], [5003], 2, 2, 48, 16, "f32", seed=6)
    # many rows of few heads: the tile kernel's split, whole, with a window, and ragged
    _attention([150], [3000], 4, 2, 128, 64, "bf16", seed=7)
    _attention([150], [3000], 4, 2, 64, 16, "bf16", window=1500, sinks=200, seed=8)
    _attention([70, 3, 200], [2500, 40, 200], 2, 1, 96, 32, "bf16", seed=9)


@pytest.mark.parametrize("batch,kv_heads,dim,dtype", [(161, 2, 64, "bf16"), (330, 1, 128, "f32"), (1027, 1, 16, "bf16")])
def test_attention_of_more_blocks_than_run_at_once(batch, kv_heads, dim, dtype):
    # sequences start in the order of their lengths: odd batches, equal lengths, empty ones,
    # and a batch above the number that is put in order
    kv = [(37 * b) % 61 * (1 + b % 3) for b in range(batch)]
    new = [min(n, 1 + (b % 11 == 0)) for b, n in enumerate(kv)]
    _attention(new, kv, 2 * kv_heads, kv_heads, dim, 16, dtype, seed=batch)


@pytest.mark.parametrize("batch,window", [(3, 0), (37, 0), (1027, 20)])
def test_attention_many_pieces(batch, window):
    # the tile kernel over sequences of different lengths, some without new tokens
    new = [[33, 0, 70, 2][b % 4] if batch < 100 or b % 257 == 0 else b % 2 for b in range(batch)]
    kv = [n + (53 * b) % 207 for b, n in enumerate(new)]
    _attention(new, kv, 12, 3, 64, 32, "bf16", window=window, seed=batch)


def test_attention_rows_that_see_nothing_are_zero():
    table, start, length, pages = ref.make_tables([1, 1, 3], [0, 5, 2], 16, width=2)
    k, v, ks, vs = _cache(0, pages, 2, 16, 64)
    cache, batch = _handles(k, v, ks, vs, table, start, length, 3)
    q = torch.randn(5, 4, 64, generator=_gen(1)).bfloat16()
    out = torch.full((5, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    caat.paged_attention(q.cuda(), cache, batch, out=out, softmax_scale=0.05)
    assert caat.device_status() == 0
    assert (out[0] == 0).all() and (out[2] == 0).all()        # no position
    want, spread = ref.attention(q, k, v, ks, vs, table, start, length, 16, 0.05)
    _check_attention(out, want, spread, "bf16")


@pytest.mark.parametrize("new", [[1, 1], [6, 3], [140, 60]])
def test_attention_stale_nan_codes_are_not_seen(new):
    def edit(q, k, v, ks, vs, table):
        # what lies behind a sequence's last token is whatever was there: NaN
        for b, n in enumerate(kv):
            if n % 32:
                pg = int(table[b, n // 32])
                k[pg, :, n % 32:] = float("nan")
                v[pg, :, n % 32:] = float("nan")
    kv = [n + p for n, p in zip(new, (35, 90))]
    got, _ = _attention(new, kv, 4, 2, 64, 32, "bf16", seed=9, edit=edit)
    assert torch.isfinite(got.float()).all()


@pytest.mark.parametrize("new,window", [([1, 1], 40), ([6, 3], 40), ([6, 3], 0), ([140, 60], 0), ([140, 60], 40)])
def test_attention_nan_reaches_only_the_rows_that_see_it(new, window):
    kv = [n + 50 for n in new]

    def edit(q, k, v, ks, vs, table):
        for b, n in enumerate(kv):
            for at, x in ((3, v), (n - 2, v), (n - 1, k)):
                x[int(table[b, at // 32]), 0, at % 32, 5] = float("nan")
    got, want = _attention(new, kv, 4, 2, 64, 32, "bf16", window=window, sinks=2, seed=11, edit=edit)
    assert torch.equal(torch.isnan(got.cpu()), torch.isnan(want))
    assert torch.isnan(want).any() and not torch.isnan(want).all()


def test_attention_scales_far_apart():
    # value scales 2^10 apart from page to page, in both orders; peaked and flat weights
    def edit(q, k, v, ks, vs, table):
        vs.copy_(torch.exp2(torch.tensor([(-5.0, 5.0)[i % 2] for i in range(vs.shape[0])]))[:, None].expand_as(vs))
        ks.fill_(2.0 ** -7)
    for new in ([1, 1], [80, 33]):
        for q_scale in (0.1, 3.0):
            _attention(new, [n + 200 for n in new], 4, 2, 64, 16, "bf16", seed=4, edit=edit, q_scale=q_scale)


def test_attention_strided_queries_and_output():
    new, kv, page, D = [3, 1, 40], [50, 9, 77], 16, 64
    table, start, length, pages = ref.make_tables(new, kv, page)
    k, v, ks, vs = _cache(2, pages, 2, page, D)
    cache, batch = _handles(k, v, ks, vs, table, start, length, 40)
    T = sum(new)
    rows = torch.randn(T, 2, 5, D, generator=_gen(3)).bfloat16()      # a cached head's 3 queries, key, value
    q4 = rows.cuda()[:, :, :3]
    buf = torch.zeros(T, 8, D, dtype=torch.bfloat16, device="cuda")
    out = caat.paged_attention(q4, cache, batch, out=buf[:, 1:7], softmax_scale=0.05)
    assert caat.device_status() == 0
    want, spread = ref.attention(rows[:, :, :3].reshape(T, 6, D), k, v, ks, vs, table, start, length, page, 0.05)
    _check_attention(out, want, spread, "bf16")
    assert (buf[:, 0] == 0).all() and (buf[:, 7] == 0).all()


def test_attention_in_a_padded_cache_of_several_layers():
    # pages of one layer lie between those of another; the offsets pass 2^31
    pages, G, page, D = 12, 1, 128, 128
    stride = (1 << 28) + G * page * D
    table, start, length, _ = ref.make_tables([2], [700], page, spare=0)
    table += 4                                                       # the last pages: offsets beyond 2^31
    k, v, ks, vs = _cache(5, pages, G, page, D)
    big = torch.empty(stride * pages, dtype=torch.uint8, device="cuda")
    kd = big.view(F8).as_strided((pages, G, page, D), (stride, page * D, D, 1))
    vd = big[G * page * D:].view(F8).as_strided((pages, G, page, D), (stride, page * D, D, 1))
    kd.view(torch.uint8).copy_(k.view(torch.uint8))
    vd.view(torch.uint8).copy_(v.view(torch.uint8))
    cache = caat.PagedKVCache(kd, vd, ks.cuda(), vs.cuda())
    batch = caat.PagedBatch(table.cuda(), start.cuda(), length.cuda(), 2)
    q = torch.randn(2, 2, D, generator=_gen(1)).bfloat16()
    got = caat.paged_attention(q.cuda(), cache, batch, softmax_scale=0.03)
    want, spread = ref.attention(q, k, v, ks, vs, table, start, length, page, 0.03)
    _check_attention(got, want, spread, "bf16")


# ------------------------------------------------------------------ append

def _append(new, kv, heads, kv_heads, dim, page, dtype, interleaved, rot, seed=0, edit=None, mag=1.0):
    table, start, length, pages = ref.make_tables(new, kv, page, seed=seed)
    k, v, ks, vs = _cache(seed + 1, pages, kv_heads, page, dim)
    T = sum(new)
    g = _gen(seed + 2)
    x = (torch.randn(T, heads + 2 * kv_heads, dim, generator=g) * mag).to(DT[dtype])
    if edit is not None:
        edit(x)
    a = torch.randn(max(kv) + 1, rot // 2, generator=g) * 3 if rot else None
    cos, sin = (a.cos(), a.sin()) if rot else (None, None)
    cache, batch = _handles(k, v, ks, vs, table, start, length, max(new))
    xd = x.cuda()
    q = caat.rope_append(xd[:, :heads], xd[:, heads:heads + kv_heads], xd[:, heads + kv_heads:],
                         cos.cuda() if rot else None, sin.cuda() if rot else None, cache, batch, interleaved=interleaved)
    assert caat.device_status() == 0
    want = ref.append(x[:, :heads], x[:, heads:heads + kv_heads], x[:, heads + kv_heads:], cos, sin, rot, interleaved,
                      k, v, ks, vs, table, start, length, page)
    assert _same_bits(q, want.to(DT[dtype]))
    assert _same_bits(cache.k_scale, ks) and _same_bits(cache.v_scale, vs)
    assert _same_bits(cache.k, k) and _same_bits(cache.v, v)
    return cache


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(16, 16), (48, 32), (64, 64), (80, 16), (128, 128), (96, 0), (128, 96)])
@pytest.mark.parametrize("page", [16, 128])
def test_append(dtype, interleaved, dim, rot, page):
    _append([1, 1, 3, 20, 140], [1, 33, 3, 77, 300], 4, 2, dim, page, dtype, interleaved, rot, seed=dim)


@pytest.mark.parametrize("new,kv", [([1], [1]), ([1, 1, 1], [16, 17, 48]), ([0, 2, 0], [5, 2, 0]), ([16, 32], [16, 64]),
                                    ([65], [200]), ([3, 2], [1, 0])])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (8, 2), (5, 5)])
def test_append_lengths(new, kv, heads, kv_heads):
    _append(new, kv, heads, kv_heads, 64, 16, "bf16", False, 64, seed=len(new))


def test_append_scale_grows_and_the_held_codes_with_it():
    # large new rows behind small ones: the held codes are brought to the larger scale,
    # some into the subnormals; and tiny ones, which leave it
    for mag in (1e-3, 1.0, 40.0, 3000.0, 1e20):
        _append([1, 2], [9, 30], 2, 2, 64, 16, "f32", False, 64, seed=8, mag=mag)
        _append([1, 40], [120, 100], 2, 2, 128, 128, "bf16", True, 128, seed=8, mag=mag)


def test_append_zeros_infinities_and_nan():
    def edit(x):
        x[0] = 0
        x[1, :, 3] = float("inf")
        x[1, :, 40] = -float("inf")
        x[2, :, 9] = float("nan")
        x[3] = float("nan")
    for new in ([4], [1, 1, 1, 1], [30]):
        kv = [n + 21 for n in new]
        # without rotation: a turned infinity meets its partner, which the reference does alike
        for rot in (0, 64):
            _append(new, kv, 2, 2, 64, 16, "f32", False, rot, seed=2, edit=edit)


def test_append_in_place_and_from_one_fused_row():
    new, kv, page, D = [2, 19], [40, 19], 16, 64
    table, start, length, pages = ref.make_tables(new, kv, page)
    k, v, ks, vs = _cache(3, pages, 2, page, D)
    cache, batch = _handles(k, v, ks, vs, table, start, length, 19)
    x = torch.randn(21, 2, 5, D, generator=_gen(4)).bfloat16()       # a cached head's 3 queries, key, value
    a = torch.randn(64, 32, generator=_gen(5))
    xd = x.cuda()
    out = caat.rope_append(xd[:, :, :3], xd[:, :, 3], xd[:, :, 4], a.cos().cuda(), a.sin().cuda(), cache, batch)
    want = ref.append(x[:, :, :3].reshape(21, 6, D), x[:, :, 3], x[:, :, 4], a.cos(), a.sin(), 64, False, k, v, ks, vs,
                      table, start, length, page)
    assert _same_bits(out, want.bfloat16()) and _same_bits(cache.k, k) and _same_bits(cache.v, v)
    assert torch.equal(xd.cpu(), x)
    # the same into the queries themselves, laid out [tokens, heads + 2 kv_heads, dim]
    y = torch.cat([x[:, :, :3].reshape(21, 6, D), x[:, :, 3], x[:, :, 4]], 1).cuda()
    caat.rope_append(y[:, :6], y[:, 6:8], y[:, 8:], a.cos().cuda(), a.sin().cuda(), cache, batch, q_out=y[:, :6])
    assert _same_bits(y[:, :6], want.bfloat16())
    assert caat.device_status() == 0


# ---------------------------------------------------------------- sampling

def _sample(z, u, temperature, top_k, top_p, min_p):
    B = z.shape[0]
    f = lambda x, t=torch.float32: torch.as_tensor(x, dtype=t).expand(B).contiguous().cuda()  # noqa: E731
    tok, lp = caat.sample_tokens(z.cuda() if not z.is_cuda else z, f(u), f(temperature), f(top_k, torch.int32), f(top_p), f(min_p))
    return tok.cpu().numpy(), lp.cpu().numpy()


def _check_samples(z, u, temperature, top_k, top_p, min_p):
    """Every token is the reference's, or the reference's for a u or top_p within 2^-18 of
    the given ones: the kernel's running sums are good to about 2^-20 of their total.
    min_p likewise, relative."""
    tok, lp = _sample(z, u, temperature, top_k, top_p, min_p)
    B = z.shape[0]
    par = [np.broadcast_to(np.asarray(x, np.float32), (B,)) for x in (u, temperature, top_k, top_p, min_p)]
    zz = z.float().cpu().numpy()
    eps = 2.0 ** -18
    for b in range(B):
        uu, tt, kk, pp, mm = (float(x[b]) for x in par)
        want, wlp = ref.sample(zz[b], uu, tt, int(kk), pp, mm)
        if tok[b] != want:
            near = {ref.sample(zz[b], min(max(uu + du, 0), 1 - 1e-12), tt, int(kk), pp if pp >= 1 else pp + dp, mm * dm)[0]
                    for du in (-eps, 0, eps) for dp in (-eps, 0, eps) for dm in (1 - eps, 1, 1 + eps)}
            assert tok[b] in near, (b, tok[b], want, near)
            continue
        if math.isinf(wlp):
            assert lp[b] == wlp
        else:
            # fp32 logits; a sum of V terms to about 2^-21, its logarithm and one rounding
            assert abs(lp[b] - wlp) <= 2.0 ** -19 + 2.0 ** -22 * abs(wlp), (b, lp[b], wlp)


@pytest.mark.parametrize("V", [1, 2, 31, 33, 100, 1023, 4099, 32000, 131071])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sample(V, dtype):
    g = _gen(V)
    B = 12
    z = (torch.randn(B, V, generator=g) * 3).to(DT[dtype])
    z[:, torch.randint(0, V, (V // 50 + 1,), generator=g)] = -math.inf
    if V < 3:
        z = torch.randn(B, V, generator=g).to(DT[dtype])
    u = torch.rand(B, generator=g).numpy()
    r = np.arange(B)
    _check_samples(z, u, np.where(r % 4 == 3, 0.0, 0.4 + 0.2 * r), np.where(r % 3 == 0, 0, 1 + 7 * r),
                   np.where(r % 2 == 0, 1.0, 0.5 + 0.04 * r), np.where(r % 5 == 0, 0.02, 0.0))


@pytest.mark.parametrize("top_k,top_p,min_p", [(0, 1.0, 0.0), (1, 1.0, 0.0), (5, 1.0, 0.0), (0, 0.0, 0.0), (0, 1e-6, 0.0),
                                               (0, 0.9, 0.0), (0, 0.999999, 0.0), (50, 0.3, 0.0), (0, 1.0, 0.5),
                                               (0, 1.0, 1.0), (2000, 0.99, 1e-4), (100000, 0.5, 0.0), (999, 2.0, 0.0)])
@pytest.mark.parametrize("shape", ["normal", "flat", "ties", "steps", "peak"])
def test_sample_filters(top_k, top_p, min_p, shape):
    B, V = 8, 1000
    g = _gen(7)
    z = {"normal": torch.randn(B, V, generator=g) * 2, "flat": torch.full((B, V), -1.25),
         "ties": torch.randint(-2, 3, (B, V), generator=g).float(),
         "steps": torch.arange(V).float().expand(B, V) % 10 * 0.1,
         "peak": torch.randn(B, V, generator=g) + 30 * (torch.arange(V) == 123)}[shape].clone()
    _check_samples(z, np.array([0, 1e-7, 0.2, 0.4, 0.5, 0.75, 0.999, 1 - 2 ** -24], np.float32), 0.8, top_k, top_p, min_p)


def test_sample_extreme_rows():
    V = 777
    low = torch.finfo(torch.float32).min
    z = torch.randn(12, V, generator=_gen(1))
    z[0] = -math.inf                                  # nothing to draw
    z[1] = math.nan
    z[2] = -math.inf
    z[2, 700] = -3.0                                  # one token left
    z[3, 5] = z[3, 600] = math.inf                    # the infinite ones share the draw
    z[4] = low                                        # all at the type's lowest value: even
    z[5, 1:] = low
    z[6, ::2] = math.nan
    z[7] = 3e38
    z[7, 9] = -3e38
    z[8] = 0.0
    z[8, ::2] = -0.0                                  # equal values
    for t in (0.0, 1e-30, 0.7, 1.0, 1e30, math.inf):
        for u in (0.0, 0.3, 0.97):
            _check_samples(z, u, t, 0, 1.0, 0.0)
            _check_samples(z, u, t, 40, 0.9, 0.0)
    tok, lp = _sample(z, 0.5, 1.0, 0, 1.0, 0.0)
    assert tok[0] == tok[1] == -1 and lp[0] == -math.inf and tok[2] == 700 and tok[3] == 600


@pytest.mark.parametrize("V", [8193, 16400, 33001])
@pytest.mark.parametrize("shape", ["flat", "ties", "steps", "peak"])
def test_sample_rows_over_several_blocks(V, shape):
    # long rows of a small batch: two, four and eight blocks a row, the last one's share short
    B = 6
    z = {"flat": torch.full((B, V), -1.25), "ties": torch.randint(-2, 3, (B, V), generator=_gen(8)).float(),
         "steps": torch.arange(V).float().expand(B, V) % 10 * 0.1,
         "peak": torch.randn(B, V, generator=_gen(9)) + 30 * (torch.arange(V) == V - 1)}[shape].clone()
    u = np.array([0, 0.2, 0.4, 0.5, 0.75, 0.999], np.float32)
    for top_k, top_p, min_p in ((0, 1.0, 0.0), (1, 1.0, 0.0), (0, 0.9, 0.0), (50, 0.3, 0.0), (700, 1.0, 0.0), (0, 1.0, 0.5),
                                (3000, 0.99, 1e-4)):
        _check_samples(z, u, 0.8, top_k, top_p, min_p)
    _check_samples(z, u, 0.0, 0, 1.0, 0.0)


@pytest.mark.parametrize("B,V,kind", [(305, 700, "mixed"), (417, 700, "mixed"), (320, 700, "costly"), (309, 700, "cheap"),
                                      (1025, 90, "mixed"), (161, 9001, "mixed")])
def test_sample_more_rows_than_run_at_once(B, V, kind):
    # rows with top-p alone start first, wherever they stand in the batch
    g = _gen(B)
    z = torch.randn(B, V, generator=g) * 2
    r = np.arange(B)
    p = {"mixed": np.where(r % 3 == 0, 0.8, 1.0), "costly": 0.7, "cheap": 1.0}[kind]
    k = {"mixed": np.where(r % 5 == 1, 20, 0), "costly": 0, "cheap": np.where(r % 2 == 0, 9, 0)}[kind]
    _check_samples(z, torch.rand(B, generator=g).numpy(), np.where(r % 7 == 6, 0.0, 0.9), k, p, 0.0)


def test_sample_extreme_rows_over_several_blocks():
    V = 40001
    low = torch.finfo(torch.float32).min
    z = torch.randn(8, V, generator=_gen(11))
    z[0] = -math.inf
    z[1] = math.nan
    z[2] = -math.inf
    z[2, V - 1] = -3.0                                # one token left, in the last block's share
    z[3, 5] = z[3, V - 7] = math.inf                  # the infinite ones share the draw
    z[4, : V - 2] = low
    z[5, :20000] = math.nan
    z[6, 100:] = -math.inf                            # whole blocks without a token
    for temp in (0.0, 0.7, 1e30):
        for top_k, top_p in ((0, 1.0), (40, 0.9), (0, 0.6)):
            if temp > 1 and top_p < 1:
                continue                              # 40001 equal weights but for rounding: no one answer
            _check_samples(z, 0.3, temp, top_k, top_p, 0.0)
    tok, lp = _sample(z, 0.9, 1.0, 0, 1.0, 0.0)
    assert tok[0] == tok[1] == -1 and lp[0] == -math.inf and tok[2] == V - 1 and tok[3] == V - 7


def test_sample_rows_with_a_stride_and_odd_alignment():
    big = torch.randn(6, 5000, generator=_gen(3)).cuda()
    for dt in (torch.float32, torch.bfloat16):
        for off in (0, 1, 3, 7):
            z = big.to(dt)[:, off:off + 4321]
            _check_samples(z, np.linspace(0, 0.99, 6, dtype=np.float32), 0.9, 30, 0.95, 0.0)


def test_sample_distribution():
    # 40000 draws of one row: frequencies within 5 standard deviations of the kept weights
    V, B = 50, 40000
    z = torch.randn(V, generator=_gen(2)) * 1.5
    u = torch.rand(B, generator=_gen(3))
    tok, _ = _sample(z.expand(B, V).contiguous(), u.numpy(), 0.9, 20, 0.95, 0.0)
    w = torch.exp(z.double() / 0.9)
    order = w.argsort(descending=True)
    keep = order[:20]
    c = w[keep].cumsum(0) / w[keep].sum()
    keep = keep[: int((c < 0.95).sum()) + 1]
    p = np.zeros(V)
    p[keep.numpy()] = (w[keep] / w[keep].sum()).numpy()
    n = np.bincount(tok, minlength=V)
    assert (np.abs(n - B * p) <= 5 * np.sqrt(B * p * (1 - p)) + 1e-9).all()


# ------------------------------------- numbers only the device sees, streams

def _small(seed=0):
    table, start, length, pages = ref.make_tables([2, 1], [20, 33], 16, seed=seed)
    k, v, ks, vs = _cache(1, pages, 2, 16, 64)
    return table, start, length, k, v, ks, vs


@pytest.mark.parametrize("what", ["page high", "page negative", "kv_len high", "kv_len negative", "q_start high",
                                  "q_start falls", "more than q_max", "position"])
def test_bad_device_numbers_are_recorded(what):
    table, start, length, k, v, ks, vs = _small()
    q_max, positions = 2, 64
    if what == "page high":
        table[1] = k.shape[0]
    elif what == "page negative":
        table[1] = -5
    elif what == "kv_len high":
        length[0] = 16 * table.shape[1] + 1
    elif what == "kv_len negative":
        length[1] = -3
    elif what == "q_start high":
        start[2] = 5
    elif what == "q_start falls":
        start[1] = 3
    elif what == "more than q_max":
        q_max = 1
    elif what == "position":
        positions = 25
    cache, batch = _handles(k, v, ks, vs, table, start, length, q_max)
    x = torch.randn(3, 8, 64, device="cuda").bfloat16()
    a = torch.zeros(positions, 32, device="cuda")
    assert caat.device_status() == 0
    caat.rope_append(x[:, :4], x[:, 4:6], x[:, 6:], a, a, cache, batch)
    assert caat.device_status() == 1
    if what != "position":
        caat.paged_attention(x[:, :4], cache, batch)
        assert caat.device_status() == 1
    assert caat.device_status() == 0


def test_calls_follow_their_stream_and_replay_in_a_graph():
    table, start, length, k, v, ks, vs = _small()
    cache, batch = _handles(k, v, ks, vs, table, start, length, 2)
    x = torch.randn(3, 8, 64, generator=_gen(2)).bfloat16().cuda()
    a = torch.randn(64, 32, generator=_gen(3)).cuda()
    z = torch.randn(2, 500, generator=_gen(4)).cuda()
    par = [torch.tensor([0.3, 0.6]).cuda(), torch.ones(2).cuda(), torch.tensor([50, 0], dtype=torch.int32).cuda(),
           torch.tensor([0.9, 0.8]).cuda(), torch.zeros(2).cuda()]

    def step():
        q = caat.rope_append(x[:, :4], x[:, 4:6], x[:, 6:], a.cos(), a.sin(), cache, batch)
        return caat.paged_attention(q, cache, batch), caat.sample_tokens(z, *par)[0]

    first = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = [t.clone() for t in step()]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    # new numbers in the same buffers
    x.copy_(torch.randn(3, 8, 64, generator=_gen(7)).bfloat16().cuda())
    batch.kv_len.copy_(torch.tensor([19, 20], dtype=torch.int32))
    graph.replay()
    got = [t.clone() for t in out]
    want = step()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert caat.device_status() == 0


def test_sample_logprob_of_a_likely_token():
    # one token far above the rest: its log probability is -log(1 + rest), and the rest must
    # not be lost beside the 1.  Each weight is good to about 2^-21, their fp32 sums (128 terms
    # a thread) to 2^-20, and so is the logarithm, relatively.
    for V, gap in ((1000, 12.0), (32000, 16.0), (32000, 20.0), (500, 30.0)):
        z = torch.randn(4, V, generator=_gen(V)).float()
        z[:, 77] = gap
        tok, lp = _sample(z, 0.5, 0.0, 0, 1.0, 0.0)
        # (a 64-bit sum that holds the 1 too is off by 2^-53 a term: 1e-5 of a rest of 7e-11)
        rest = (z.double() - gap).exp()
        rest[:, 77] = 0.0
        want = -torch.log1p(rest.sum(-1)).numpy()
        assert (tok == 77).all() and (np.abs(lp - want) <= 2.0 ** -18 * np.abs(want)).all(), (V, gap, lp, want)
