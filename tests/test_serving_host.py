"""Refusals of the serving calls, without a GPU: fake device addresses that are never
read, each call wrong in one argument."""
import ctypes

import pytest

P0 = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from partial_activation_sync_gb300 import build
    build.build()
    from partial_activation_sync_gb300 import _lib
    return _lib.load()


def _kv(**kw):
    from partial_activation_sync_gb300 import _lib
    # 8 pages of 16 tokens, 2 heads of 64
    d = dict(k=P0, v=2 * P0, k_scale=3 * P0, v_scale=4 * P0, pages=8, page_stride=2048, scale_stride=2, kv_heads=2,
             page=16, dim=64)
    d.update(kw)
    return _lib.PagedKV(**d)


def _batch(**kw):
    from partial_activation_sync_gb300 import _lib
    d = dict(page_table=5 * P0, q_start=6 * P0, kv_len=7 * P0, table_stride=4, tokens=3, batch=2, table_width=4, q_max=2)
    d.update(kw)
    return _lib.PagedBatch(**d)


BAD_KV = [dict(k=None), dict(v=0), dict(k_scale=None), dict(v_scale=None), dict(k=P0 + 8), dict(pages=0), dict(kv_heads=0),
          dict(page=8), dict(page=48), dict(page=256), dict(dim=0), dict(dim=72), dict(dim=144), dict(page_stride=2047),
          dict(page_stride=2056), dict(scale_stride=1), dict(kv_heads=3)]
BAD_BATCH = [dict(page_table=None), dict(q_start=None), dict(kv_len=None), dict(table_stride=3), dict(tokens=-1),
             dict(batch=-1), dict(q_max=-1), dict(table_width=-1), dict(table_width=1 << 27, table_stride=1 << 27)]


def _append(lib, kv=None, batch=None, **kw):
    a = dict(heads=4, dt=1, q=8 * P0, q_st=256, q_sk=128, q_sg=64, k=9 * P0, k_st=128, k_sh=64, v=10 * P0, v_st=128,
             v_sh=64, cos=11 * P0, sin=12 * P0, positions=64, rot=64, inter=0, qo=13 * P0, qo_st=256, qo_sh=64, s=None)
    a.update(kw)
    kv, batch = kv or _kv(), batch or _batch()
    return lib.caat_rope_append(ctypes.byref(kv), ctypes.byref(batch), *a.values())


@pytest.mark.parametrize("bad", BAD_KV, ids=str)
def test_append_refuses_a_bad_cache(lib, bad):
    assert _append(lib, kv=_kv(**bad)) == 1


@pytest.mark.parametrize("bad", BAD_BATCH, ids=str)
def test_append_refuses_a_bad_batch(lib, bad):
    assert _append(lib, batch=_batch(**bad)) == 1


@pytest.mark.parametrize("bad", [
    dict(heads=3), dict(heads=0), dict(dt=2), dict(q=None), dict(k=None), dict(v=None), dict(qo=None), dict(cos=None),
    dict(sin=None), dict(cos=11 * P0 + 4), dict(q=8 * P0 + 2), dict(q_st=-256), dict(q_st=252), dict(k_sh=65),
    dict(v_st=4), dict(qo_sh=63), dict(qo_sh=0), dict(qo_st=0), dict(qo_st=64), dict(rot=24), dict(rot=-16),
    dict(rot=80), dict(positions=0), dict(qo=9 * P0), dict(qo=10 * P0 + 128), dict(qo=8 * P0 + 64), dict(qo=11 * P0 + 64),
    dict(qo=P0 + 64), dict(k=2 * P0), dict(qo=5 * P0), dict(qo=4 * P0), dict(qo=8 * P0, qo_st=512)], ids=str)
def test_append_refuses_bad_arguments(lib, bad):
    assert _append(lib, **bad) == 1


def _attention(lib, kv=None, batch=None, **kw):
    a = dict(heads=4, dt=1, q=8 * P0, q_st=256, q_sk=128, q_sg=64, scale=0.1, window=0, sinks=0, o=13 * P0, o_st=256,
             o_sh=64, s=None)
    a.update(kw)
    kv, batch = kv or _kv(), batch or _batch()
    return lib.caat_paged_attention(ctypes.byref(kv), ctypes.byref(batch), *a.values())


@pytest.mark.parametrize("bad", BAD_KV, ids=str)
def test_attention_refuses_a_bad_cache(lib, bad):
    assert _attention(lib, kv=_kv(**bad)) == 1


@pytest.mark.parametrize("bad", BAD_BATCH, ids=str)
def test_attention_refuses_a_bad_batch(lib, bad):
    assert _attention(lib, batch=_batch(**bad)) == 1


@pytest.mark.parametrize("bad", [
    dict(heads=5), dict(dt=7), dict(q=None), dict(o=None), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(window=-1), dict(sinks=-1), dict(q=8 * P0 + 8), dict(o=13 * P0 + 8), dict(o_st=100),
    dict(o_sh=0), dict(o=8 * P0), dict(o=P0), dict(o=2 * P0 + 64), dict(o=3 * P0), dict(o=5 * P0), dict(o=6 * P0),
    dict(o=7 * P0)], ids=str)
def test_attention_refuses_bad_arguments(lib, bad):
    assert _attention(lib, **bad) == 1


def _sample(lib, **kw):
    a = dict(batch=2, vocab=100, dt=0, logits=P0, ld=100, u=2 * P0, t=3 * P0, k=4 * P0, p=5 * P0, m=6 * P0, tok=7 * P0,
             lp=8 * P0, s=None)
    a.update(kw)
    return lib.caat_sample_tokens(*a.values())


@pytest.mark.parametrize("bad", [
    dict(batch=-1), dict(vocab=0), dict(vocab=1 << 31, ld=1 << 31), dict(ld=99), dict(dt=3), dict(logits=None), dict(u=None),
    dict(t=None), dict(k=None), dict(p=None), dict(m=None), dict(tok=None), dict(lp=None), dict(tok=8 * P0),
    dict(lp=P0 + 400), dict(tok=2 * P0 + 4)], ids=str)
def test_sample_refuses_bad_arguments(lib, bad):
    assert _sample(lib, **bad) == 1


def test_null_handles_are_refused(lib):
    assert lib.caat_rope_append(None, None, 4, 1, *([8 * P0, 256, 128, 64] + [9 * P0, 128, 64] + [10 * P0, 128, 64]),
                                11 * P0, 12 * P0, 64, 64, 0, 13 * P0, 256, 64, None) == 1
    assert lib.caat_paged_attention(None, ctypes.byref(_batch()), 4, 1, 8 * P0, 256, 128, 64, 0.1, 0, 0, 13 * P0, 256, 64,
                                    None) == 1


def test_work_of_nothing_is_no_error(lib):
    assert _append(lib, batch=_batch(tokens=0)) == 0
    assert _append(lib, batch=_batch(batch=0)) == 0
    assert _attention(lib, batch=_batch(q_max=0)) == 0
    assert _sample(lib, batch=0) == 0


def test_handles_refuse_what_does_not_fit():
    import torch

    import partial_activation_sync_gb300 as caat
    f8 = torch.float8_e4m3fn
    k = torch.zeros(4, 2, 16, 64, dtype=f8)
    s = torch.ones(4, 2)
    with pytest.raises(ValueError, match="CUDA"):
        caat.PagedKVCache(k, k, s, s)                    # not on a GPU
    for shape in ((4, 2, 16), (4, 2, 24, 64), (4, 2, 16, 40), (4, 2, 16, 256)):
        with pytest.raises(ValueError):
            caat.PagedKVCache(torch.zeros(shape, dtype=f8), k, s, s)
    with pytest.raises(ValueError, match="page_table"):
        caat.PagedBatch(torch.zeros(2, 4), None, None, 1)
    with pytest.raises(ValueError):
        caat.sample_tokens(torch.zeros(4), None, None, None, None, None)
