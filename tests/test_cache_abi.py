"""Refusals of the cache's entry points on the host (no GPU needed): bad
arguments are rejected before the device is touched."""

import ctypes

import pytest
import torch

from exact_attention_fattn_gb300 import _lib, cache
from test_abi import lib  # noqa: F401  (fixture)

GOOD = 0x10000   # a 256-byte aligned fake address; never dereferenced


def _cache(**kw):
    a = dict(k=GOOD, v=GOOD, k_scale=GOOD, v_scale=GOOD, k_bounds=GOOD, page_stride=2 * 64 * 128, pages=4, Hkv=2,
             page=64, d=128)
    a.update(kw)
    return _lib.CacheStruct(*(a[n] for n, _ in _lib.CacheStruct._fields_))


BAD_CACHES = [
    (dict(k=0), 1), (dict(v=GOOD + 8), 1), (dict(k_scale=0), 1), (dict(v_scale=GOOD + 2), 1), (dict(pages=0), 1),
    (dict(Hkv=0), 1), (dict(Hkv=1025, page_stride=1 << 30), 1), (dict(page=16), 2), (dict(page=48), 2), (dict(d=96), 2),
    (dict(page_stride=2 * 64 * 128 - 16), 1), (dict(page_stride=2 * 64 * 128 + 8), 1), (dict(page_stride=1 << 40), 1),
]


def _append(lib, c, **kw):
    a = dict(k_new=GOOD, k_row=256, v_new=GOOD, v_row=256, q=GOOD, q_row=1024, q_out=GOOD + 4096, Hq=8, rope=GOOD,
             rope_len=100, rope_dim=128, interleaved=0, page_table=GOOD, q_start=GOOD, kv_len=GOOD, T=3, B=2, max_pages=2)
    a.update(kw)
    return lib.fattn_cache_append(ctypes.byref(c) if c else None, *a.values(), None)


def _fwd(lib, c, **kw):
    a = dict(q=GOOD, q_row=1024, o=GOOD, lse=GOOD, page_table=GOOD, q_start=GOOD, kv_len=GOOD, selected=0, n_selected=0,
             ws=GOOD, ws_bytes=1 << 40, T=3, B=2, Hq=8, max_pages=2, causal=1, scale=0.1)
    a.update(kw)
    return lib.fattn_cache_fwd(ctypes.byref(c) if c else None, *a.values(), None)


def _select(lib, c, **kw):
    a = dict(q=GOOD, q_row=1024, page_table=GOOD, q_start=GOOD, kv_len=GOOD, selected=GOOD, n_selected=4, n_first=1,
             n_recent=1, ws=GOOD, ws_bytes=1 << 40, T=3, B=2, Hq=8, max_pages=2)
    a.update(kw)
    return lib.fattn_cache_select(ctypes.byref(c) if c else None, *a.values(), None)


@pytest.mark.parametrize("kw,want", BAD_CACHES)
@pytest.mark.parametrize("call", [_append, _fwd, _select])
def test_bad_cache(lib, call, kw, want):  # noqa: F811
    assert call(lib, _cache(**kw)) == want
    assert call(lib, None) == 1


BAD_BATCH = [dict(page_table=0), dict(q_start=0), dict(kv_len=GOOD + 2), dict(T=0), dict(B=0), dict(B=4097),
             dict(max_pages=0), dict(max_pages=1 << 26), dict(Hq=7), dict(Hq=0), dict(Hq=2 * 129, q_row=1 << 20),
             dict(T=1 << 29), dict(q_row=1016), dict(q_row=1028), dict(q=GOOD + 8)]


@pytest.mark.parametrize("kw", BAD_BATCH)
@pytest.mark.parametrize("call", [_append, _fwd, _select])
def test_bad_batch(lib, call, kw):  # noqa: F811
    assert call(lib, _cache(), **kw) == 1


@pytest.mark.parametrize("kw", [
    dict(k_new=0), dict(v_new=GOOD + 2), dict(k_row=248), dict(v_row=260), dict(q=0), dict(q_out=0), dict(q_out=GOOD + 8),
    dict(q=GOOD, q_out=GOOD, q_row=1536), dict(rope=0), dict(rope=GOOD + 4), dict(rope_dim=0), dict(rope_dim=24),
    dict(rope_dim=144), dict(rope_len=0)])
def test_bad_append(lib, kw):  # noqa: F811
    assert _append(lib, _cache(), **kw) == 1


def test_bad_fwd(lib):  # noqa: F811
    need = lib.fattn_cache_fwd_workspace_bytes(3, 2, 8, 2, 128, 0)
    assert need > 0
    for kw in (dict(o=0), dict(o=GOOD + 8), dict(lse=0), dict(lse=GOOD + 2), dict(scale=0.0), dict(scale=float("nan")),
               dict(scale=-1.0), dict(selected=GOOD), dict(n_selected=4), dict(selected=GOOD, n_selected=-1),
               dict(selected=GOOD + 2, n_selected=4), dict(selected=GOOD, n_selected=1 << 26), dict(ws=0),
               dict(ws=GOOD + 16), dict(ws_bytes=need - 1)):
        assert _fwd(lib, _cache(), **kw) == 1, kw
    for bad in ((0, 1, 8, 2, 128, 0), (3, 0, 8, 2, 128, 0), (3, 5000, 8, 2, 128, 0), (3, 1, 7, 2, 128, 0),
                (3, 1, 8, 2, 96, 0), (3, 1, 8, 2, 128, -1), (3, 1, 258, 2, 128, 0)):
        assert lib.fattn_cache_fwd_workspace_bytes(*bad) == 0


def test_bad_select(lib):  # noqa: F811
    # Sizes whose scores stay on chip need no workspace; many pages do.
    assert lib.fattn_cache_select_workspace_bytes(3, 2, 2) == 256
    need = lib.fattn_cache_select_workspace_bytes(3, 2, 20000)
    assert need >= 3 * 2 * 20000 * 4
    assert _select(lib, _cache(k_bounds=0)) == 1
    assert _select(lib, _cache(k_bounds=GOOD + 8)) == 1
    for kw in (dict(selected=0), dict(selected=GOOD + 2), dict(n_selected=0), dict(n_first=-1), dict(n_recent=-1),
               dict(n_first=3, n_recent=2), dict(ws=0, max_pages=20000), dict(ws=GOOD + 16, max_pages=20000),
               dict(ws_bytes=need - 1, max_pages=20000)):
        assert _select(lib, _cache(), **kw) == 1, kw
    assert lib.fattn_cache_select_workspace_bytes(0, 2, 2) == 0
    assert lib.fattn_cache_select_workspace_bytes(3, 2, 0) == 0


def test_status_string(lib):  # noqa: F811
    assert b"out of range" in lib.fattn_status_string(_lib.FATTN_ERR_BAD_INDEX)


def test_helpers_refuse():
    for kw in (dict(pages=0), dict(page=16), dict(d=96), dict(kv_heads=0)):
        a = dict(pages=2, kv_heads=1, d=64, page=32, device="cpu")
        a.update(kw)
        with pytest.raises(ValueError):
            cache.fattn_cache_alloc(**a)
    for args in ((0, 32), (4, 8), (4, 24)):
        with pytest.raises(ValueError):
            cache.fattn_rope_table(*args, device="cpu")
    t = cache.fattn_rope_table(200001, 32, device="cpu")
    ang = 200000.0 * 10000.0 ** (-2 * 3 / 32)
    assert abs(float(t[200000, 3]) - __import__("math").cos(ang)) < 1e-7
    c = cache.fattn_cache_alloc(2, 1, 64, page=32, device="cpu", bounds=True)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        cache.fattn_cache_fwd(torch.zeros((1, 1, 64), dtype=torch.bfloat16), c, i.view(1, 2), i, i[:1])
