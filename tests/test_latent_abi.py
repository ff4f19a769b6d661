"""Refusals of the latent cache's, the pages' and the rotation's entry points on
the host (no GPU needed): bad arguments are rejected before the device is
touched."""

import ctypes

import pytest
import torch

import exact_attention_fattn_gb300 as F
from exact_attention_fattn_gb300 import _lib
from test_abi import lib  # noqa: F401  (fixture)

GOOD = 0x10000   # a 256-byte aligned fake address; never dereferenced


def _latent(**kw):
    a = dict(data=GOOD, page_stride=64 * 576, pages=4, page=64, rank=512)
    a.update(kw)
    return _lib.LatentCacheStruct(*(a[n] for n, _ in _lib.LatentCacheStruct._fields_))


def _append(lib, c, **kw):
    a = dict(latent=GOOD, latent_row=576, k_rope=GOOD, k_row=576, q_rope=GOOD, q_row=8 * 192, q_head=192, q=GOOD, Hq=8,
             rope=GOOD, rope_len=100, interleaved=0, page_table=GOOD, q_start=GOOD, kv_len=GOOD, T=3, B=2, max_pages=2)
    a.update(kw)
    return lib.fattn_latent_append(ctypes.byref(c) if c else None, *a.values(), None)


def _fwd(lib, c, **kw):
    a = dict(q=GOOD, o=GOOD, lse=GOOD, page_table=GOOD, q_start=GOOD, kv_len=GOOD, ws=GOOD, ws_bytes=1 << 40, T=3, B=2, Hq=8,
             max_pages=2, causal=1, scale=0.1)
    a.update(kw)
    return lib.fattn_latent_fwd(ctypes.byref(c) if c else None, *a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(data=0), 1), (dict(data=GOOD + 8), 1), (dict(pages=0), 1), (dict(page=16), 2), (dict(page=256), 2),
    (dict(rank=128), 2), (dict(rank=576), 2), (dict(page_stride=64 * 576 - 8), 1), (dict(page_stride=64 * 576 + 4), 1),
    (dict(page_stride=1 << 38), 1)])
@pytest.mark.parametrize("call", [_append, _fwd])
def test_bad_cache(lib, call, kw, want):  # noqa: F811
    assert call(lib, _latent(**kw)) == want
    assert call(lib, None) == 1


@pytest.mark.parametrize("kw", [
    dict(page_table=0), dict(q_start=0), dict(kv_len=GOOD + 2), dict(T=0), dict(B=0), dict(B=4097), dict(max_pages=0),
    dict(max_pages=1 << 26), dict(Hq=0), dict(Hq=1025), dict(T=1 << 29)])
@pytest.mark.parametrize("call", [_append, _fwd])
def test_bad_batch(lib, call, kw):  # noqa: F811
    assert call(lib, _latent(), **kw) == 1


@pytest.mark.parametrize("kw", [
    dict(latent=0), dict(latent=GOOD + 8), dict(latent_row=504), dict(latent_row=516), dict(k_rope=0), dict(k_row=56),
    dict(k_row=68), dict(q_rope=0), dict(q=0), dict(q=GOOD + 8), dict(q_rope=GOOD + 8), dict(q_head=56), dict(q_head=196),
    dict(q_row=56), dict(q_row=1540), dict(rope=GOOD + 4), dict(rope_len=0), dict(latent_row=1 << 32)])
def test_bad_append(lib, kw):  # noqa: F811
    assert _append(lib, _latent(), **kw) == 1


def test_bad_fwd(lib):  # noqa: F811
    need = lib.fattn_latent_fwd_workspace_bytes(3, 2, 8, 512)
    assert need > 0
    for kw in (dict(q=0), dict(q=GOOD + 8), dict(o=0), dict(o=GOOD + 8), dict(lse=0), dict(lse=GOOD + 2), dict(scale=0.0),
               dict(scale=float("nan")), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=3e38), dict(ws=0),
               dict(ws=GOOD + 16), dict(ws_bytes=need - 1)):
        assert _fwd(lib, _latent(), **kw) == 1, kw
    for bad in ((0, 1, 8, 512), (3, 0, 8, 512), (3, 4097, 8, 512), (3, 1, 0, 512), (3, 1, 8, 384), (3, 1, 1025, 512),
                (1 << 30, 1, 8, 512)):
        assert lib.fattn_latent_fwd_workspace_bytes(*bad) == 0


def _rope(lib, **kw):
    a = dict(x=GOOD, x_b=8 * 4 * 64, x_h=4 * 64, x_n=64, y=GOOD + 65536, y_b=8 * 4 * 64, y_h=4 * 64, y_n=64, rope=GOOD,
             rope_len=10, rope_dim=64, interleaved=0, transposed=0, positions=GOOD, positions_b=4, B=2, H=8, N=4, d=64)
    a.update(kw)
    return lib.fattn_rope(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(d=0), 2), (dict(d=72), 2), (dict(d=1040), 2), (dict(x=0), 1), (dict(y=0), 1), (dict(rope=0), 1), (dict(x=GOOD + 8), 1),
    (dict(y=GOOD + 8), 1), (dict(rope=GOOD + 8), 1), (dict(positions=GOOD + 2), 1), (dict(B=0), 1), (dict(H=0), 1),
    (dict(N=-1), 1), (dict(rope_len=0), 1), (dict(rope_dim=0), 1), (dict(rope_dim=24), 1), (dict(rope_dim=80), 1),
    (dict(positions_b=-1), 1), (dict(x_n=-64), 1), (dict(x_n=68), 1), (dict(x_b=1 << 40), 1),
    # rows of y that overlap: broadcast, closer than they are long, or two strides that meet
    (dict(y_b=0), 1), (dict(y_n=56), 1), (dict(y_h=64, y_n=64), 1), (dict(y_h=128, y_n=64), 1),
    # in place with other distances
    (dict(y=GOOD, y_n=512, y_h=64), 1), (dict(y=GOOD, x_h=0), 1)])
def test_bad_rope(lib, kw, want):  # noqa: F811
    assert _rope(lib, **kw) == want


def _pool(**kw):
    a = dict(refs=GOOD, pages=10, page=64)
    a.update(kw)
    return _lib.PagePoolStruct(a["refs"], a["pages"], a["page"])


def _planes(*planes):
    return (_lib.PlaneStruct * len(planes))(*planes)


ONE = (GOOD, 4096, 4096)


def _fork(lib, pool, **kw):
    a = dict(table=GOOD, kv_len=GOOD, parent=GOOD, child=GOOD, n=2, B=4, max_pages=3)
    a.update(kw)
    return lib.fattn_pages_fork(ctypes.byref(pool) if pool else None, *a.values(), None)


def _free(lib, pool, **kw):
    a = dict(table=GOOD, kv_len=GOOD, rows=GOOD, n=2, B=4, max_pages=3)
    a.update(kw)
    return lib.fattn_pages_free(ctypes.byref(pool) if pool else None, *a.values(), None)


def _extend(lib, pool, planes=None, **kw):
    planes = _planes(ONE) if planes is None else planes
    a = dict(n_planes=len(planes), table=GOOD, kv_len=GOOD, new=GOOD, ws=GOOD, ws_bytes=1 << 30, B=4, max_pages=3)
    a.update(kw)
    return lib.fattn_pages_extend(ctypes.byref(pool) if pool else None, planes, *a.values(), None)


def _compact(lib, pool, planes=None, **kw):
    planes = _planes(ONE) if planes is None else planes
    a = dict(n_planes=len(planes), table=GOOD, kv_len=GOOD, ws=GOOD, ws_bytes=1 << 30, B=4, max_pages=3)
    a.update(kw)
    return lib.fattn_pages_compact(ctypes.byref(pool) if pool else None, planes, *a.values(), None)


@pytest.mark.parametrize("call", [_fork, _free, _extend, _compact])
def test_bad_pool_and_table(lib, call):  # noqa: F811
    assert call(lib, None) == 1
    for kw, want in ((dict(refs=0), 1), (dict(refs=GOOD + 2), 1), (dict(pages=0), 1), (dict(pages=1 << 30), 1),
                     (dict(page=16), 2), (dict(page=65), 2)):
        assert call(lib, _pool(**kw)) == want, kw
    for kw in (dict(table=0), dict(table=GOOD + 2), dict(kv_len=0), dict(kv_len=GOOD + 1), dict(B=0), dict(B=4097),
               dict(max_pages=0), dict(max_pages=1 << 26)):
        assert call(lib, _pool(), **kw) == 1, kw


def test_bad_lists(lib):  # noqa: F811
    for kw in (dict(parent=0), dict(child=0), dict(child=GOOD + 2), dict(n=0), dict(n=5)):
        assert _fork(lib, _pool(), **kw) == 1, kw
    for kw in (dict(rows=0), dict(rows=GOOD + 2), dict(n=0), dict(n=4097)):
        assert _free(lib, _pool(), **kw) == 1, kw


@pytest.mark.parametrize("call", [_extend, _compact])
def test_bad_planes_and_workspace(lib, call):  # noqa: F811
    for plane in ((0, 4096, 4096), (GOOD + 2, 4096, 4096), (GOOD, 4092, 4096), (GOOD, 4098, 4096), (GOOD, 4096, 4094),
                  (GOOD, 4096, 0), (GOOD, 1 << 40, 4096), (GOOD, 1 << 39, 1 << 31)):
        assert call(lib, _pool(), _planes(ONE, plane)) == 1, plane
    assert call(lib, _pool(), n_planes=0) == 1
    assert call(lib, _pool(), _planes(*[ONE] * 6)) == 1
    need = lib.fattn_pages_workspace_bytes(10, 4)
    for kw in (dict(ws=0), dict(ws=GOOD + 16), dict(ws_bytes=need - 1)):
        assert call(lib, _pool(), **kw) == 1, kw
    for bad in ((0, 4), (10, 0), (10, 4097), (1 << 30, 4)):
        assert lib.fattn_pages_workspace_bytes(*bad) == 0
    if call is _extend:
        assert _extend(lib, _pool(), new=0) == 1 and _extend(lib, _pool(), new=GOOD + 2) == 1


def test_status_string(lib):  # noqa: F811
    assert b"free pages" in lib.fattn_status_string(_lib.FATTN_ERR_NO_PAGES)


def test_helpers_refuse():
    for kw in (dict(pages=0), dict(page=16), dict(rank=128)):
        a = dict(pages=2, rank=256, page=32, device="cpu")
        a.update(kw)
        with pytest.raises(ValueError):
            F.fattn_latent_alloc(**a)
    c = F.fattn_latent_alloc(2, 256, page=32, device="cpu")
    assert c.data.shape == (2, 32, 320) and F.fattn_pages_alloc(c).refs.tolist() == [0, 0]
    i = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros((1, 1, 320), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        F.fattn_latent_fwd(q, c, i.view(1, 2), i, i[:1], scale=1.0)
    with pytest.raises(ValueError):
        F.fattn_latent_append(q[0, :, :256], q[0, :, :64], c, i.view(1, 2), i, i[:1])
    with pytest.raises(ValueError):
        F.fattn_rope(q, F.fattn_rope_table(4, 32, device="cpu"))
    with pytest.raises(ValueError):
        F.fattn_pages_extend(F.fattn_pages_alloc(c), c, i.view(1, 2), i[:1], i[:1])
    with pytest.raises(TypeError):
        F.fattn_pages_alloc(c.data)
