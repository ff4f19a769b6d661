"""Python entry points for the pages of a cache: sequences that share pages, and
the pool that they come from, with the C ABI's names."""

from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

import torch

from . import _lib
from .cache import (PAGE_SIZES, Fp8Cache, _call, _check_cache, _current_device, _raw_alloc, _raw_free, _raw_stream,
                    _workspace)
from .latent import LatentCache, _check_latent


class PagePool(NamedTuple):
    """How many table entries name each page; a page is free while its count is 0."""

    refs: torch.Tensor      # int32 [pages]


def fattn_pages_alloc(cache) -> PagePool:
    """The pool of an empty cache's pages, all free."""
    pages = _data(cache).shape[0]
    return PagePool(torch.zeros(pages, dtype=torch.int32, device=_data(cache).device))


def _data(cache):
    if isinstance(cache, LatentCache):
        return cache.data
    if isinstance(cache, Fp8Cache):
        return cache.k
    raise TypeError("cache must be an Fp8Cache or a LatentCache")


def _setup(pool, cache, page_table, *lens):
    """The C ABI's descriptions of the pool and the cache's planes, with the device
    index and the table's shape."""
    if isinstance(cache, LatentCache):
        cs, dev = _check_latent(cache)
        page = cs.page
        planes = [(cs.data, 2 * cs.page_stride, 2 * page * (cs.rank + 64))]
    elif isinstance(cache, Fp8Cache):
        cs, dev = _check_cache(cache)
        page = cs.page
        size = cs.Hkv * page * cs.d
        planes = [(cs.k, cs.page_stride, size), (cs.v, cs.page_stride, size), (cs.k_scale, 4 * cs.Hkv, 4 * cs.Hkv),
                  (cs.v_scale, 4 * cs.Hkv, 4 * cs.Hkv)]
        if cs.k_bounds:
            planes.append((cs.k_bounds, 2 * cs.Hkv * cs.d, 2 * cs.Hkv * cs.d))
    else:
        raise TypeError("cache must be an Fp8Cache or a LatentCache")
    if page not in PAGE_SIZES:
        raise ValueError("a page must have 32, 64 or 128 tokens")
    refs = pool.refs
    if refs.dtype is not torch.int32 or refs.shape != (cs.pages,) or refs.get_device() != dev or not refs.is_contiguous():
        raise ValueError("the pool must count the cache's pages (contiguous int32 [pages] on its device)")
    shape = page_table.shape
    if page_table.dtype is not torch.int32 or len(shape) != 2 or page_table.get_device() != dev or not page_table.is_contiguous():
        raise ValueError("page_table must be a contiguous int32 [B, max_pages] tensor on the cache's device")
    for t in lens:
        if t.dtype is not torch.int32 or t.shape != shape[:1] or t.get_device() != dev or not t.is_contiguous():
            raise ValueError("lengths must be contiguous int32 [B] tensors on the cache's device")
    arr = (_lib.PlaneStruct * len(planes))(*planes)
    return _lib.PagePoolStruct(refs.data_ptr(), cs.pages, page), arr, dev, shape


def _index(t, name, dev):
    if t.dtype is not torch.int32 or t.dim() != 1 or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 [n] tensor on the cache's device")
    return t.shape[0]


@functools.lru_cache(maxsize=1024)
def fattn_pages_workspace_bytes(pages: int, B: int) -> int:
    return int(_lib.load().fattn_pages_workspace_bytes(pages, B))


def _with_workspace(fn, ps, dev, workspace, page_table, before, after):
    """fn(pool, *before, workspace, its bytes, *after)."""
    need = fattn_pages_workspace_bytes(ps.pages, page_table.shape[0])
    scratch = 0
    if workspace is None and need and _raw_alloc and _raw_free and _current_device() == dev:
        # as in fattn_cache_fwd: a block that the stream's next calls may have
        scratch = ws_ptr = _raw_alloc(need, _raw_stream(dev))
    else:
        ws = _workspace(workspace, need, page_table.device, dev)
        ws_ptr, need = ws.data_ptr(), ws.numel()
    try:
        _call(fn, dev, ctypes.byref(ps), *before, ws_ptr, need, *after)
    finally:
        if scratch:
            _raw_free(scratch)


def fattn_pages_fork(pool: PagePool, cache, page_table, kv_len, parent, child):
    """Sequence child[i] (int32 [n], of length 0) becomes a copy of sequence
    parent[i]: its table entries, its length, and its pages counted once more.
    ``page_table`` [B, max_pages] and ``kv_len`` [B] are changed."""
    ps, _, dev, (B, max_pages) = _setup(pool, cache, page_table, kv_len)
    n = _index(parent, "parent", dev)
    if _index(child, "child", dev) != n:
        raise ValueError("parent and child must have one length")
    if n == 0:
        return
    _call(_lib.load().fattn_pages_fork, dev, ctypes.byref(ps), page_table.data_ptr(), kv_len.data_ptr(), parent.data_ptr(),
          child.data_ptr(), n, B, max_pages)


def fattn_pages_extend(pool: PagePool, cache, page_table, old_len, new_len, workspace=None):
    """Make room in every sequence for its tokens old_len .. new_len - 1 (int32
    [B]), before they are appended: a copy of its last page where that is shared
    and written to, then the pages it lacks, lowest free ones first.  Changes
    ``page_table``, the counts and the copies; lengths stay.  With too few free
    pages nobody gets any, fattn_check_status() returns 8, and ``new_len`` is -1
    for the sequences that lack room (they still have ``old_len`` tokens): append
    and attention with it pass over them and serve the others."""
    ps, planes, dev, (B, max_pages) = _setup(pool, cache, page_table, old_len, new_len)
    _with_workspace(_lib.load().fattn_pages_extend, ps, dev, workspace, page_table,
                    (planes, len(planes), page_table.data_ptr(), old_len.data_ptr(), new_len.data_ptr()), (B, max_pages))


def fattn_pages_free(pool: PagePool, cache, page_table, kv_len, rows):
    """The sequences ``rows`` (int32 [n]) give their pages back; their lengths
    become 0."""
    ps, _, dev, (B, max_pages) = _setup(pool, cache, page_table, kv_len)
    n = _index(rows, "rows", dev)
    if n == 0:
        return
    _call(_lib.load().fattn_pages_free, dev, ctypes.byref(ps), page_table.data_ptr(), kv_len.data_ptr(), rows.data_ptr(), n,
          B, max_pages)


def fattn_pages_compact(pool: PagePool, cache, page_table, kv_len, workspace=None):
    """Move the pages that are held to the lowest ones, in the cache, the counts
    and the table.  ``kv_len`` says how many entries each sequence holds: the
    lengths that room was made for; with one out of range nothing moves."""
    ps, planes, dev, (B, max_pages) = _setup(pool, cache, page_table, kv_len)
    _with_workspace(_lib.load().fattn_pages_compact, ps, dev, workspace, page_table,
                    (planes, len(planes), page_table.data_ptr(), kv_len.data_ptr()), (B, max_pages))
