"""Python entry points of the paged latent cache, with the C ABI's names; as in
cache.py, they check what the host can see and hand pointers on."""

from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

import torch

from . import _lib
from .cache import (PAGE_SIZES, _call, _check_batch, _check_like, _current_device, _raw_alloc, _raw_free, _raw_stream,
                    _workspace)

ROPE = 64               # columns of the rotated key part
RANKS = (256, 512)


class LatentCache(NamedTuple):
    """A caller-owned cache: a token's latent vector and its rotated key part."""

    data: torch.Tensor      # bf16 [pages, page, rank + 64]
    rank: int


def fattn_latent_alloc(pages: int, rank: int = 512, page: int = 64, device="cuda") -> LatentCache:
    """An empty cache of ``pages`` pages of ``page`` tokens."""
    if pages < 1 or page not in PAGE_SIZES or rank not in RANKS:
        raise ValueError("need pages >= 1, page in (32, 64, 128) and rank in (256, 512)")
    return LatentCache(torch.zeros((pages, page, rank + ROPE), dtype=torch.bfloat16, device=device), rank)


def _check_latent(c: LatentCache):
    """The C ABI's description of the cache and its device index."""
    t, rank = c
    shape, dev = t.shape, t.get_device()
    if dev < 0:
        raise ValueError("libfattn works on CUDA tensors; move the cache to the GPU first")
    if t.dtype is not torch.bfloat16:
        raise TypeError("cache data must be bfloat16")
    if len(shape) != 3 or shape[2] != rank + ROPE:
        raise ValueError("cache data must be [pages, page, rank + 64]")
    s = t.stride()
    if s[2] != 1 or s[1] != shape[2]:
        raise ValueError("cache pages must be contiguous")
    return _lib.LatentCacheStruct(t.data_ptr(), s[0] if shape[0] > 1 else shape[1] * shape[2], shape[0], shape[1], rank), dev


def _check_part(t, name, columns, dev):
    """bf16 [T, columns] whose rows may lie apart: (T, their distance)."""
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    shape, s = t.shape, t.stride()
    if len(shape) != 2 or shape[1] != columns or s[1] != 1:
        raise ValueError(f"{name} must be [T, {columns}] with contiguous rows")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the cache's device")
    return shape[0], s[0] if shape[0] > 1 else columns


def fattn_latent_append(latent, k_rope, cache: LatentCache, page_table, q_start, kv_len, rope=None, q_rope=None, q=None,
                        interleaved: bool = False):
    """Append new tokens, latents (bf16 [T, rank]) and key parts (bf16 [T, 64],
    rotated by ``rope``), to their sequences' pages.  With ``q_rope`` (bf16 [T,
    Hq, 64], may be strided) the queries' parts are rotated into the last 64
    columns of ``q`` (bf16 [T, Hq, rank + 64]), which is returned.  The batch is
    described as for fattn_cache_append."""
    cs, dev = _check_latent(cache)
    B, max_pages = _check_batch(page_table, q_start, kv_len, dev)
    T, latent_row = _check_part(latent, "latent", cs.rank, dev)
    Tk, k_row = _check_part(k_rope, "k_rope", ROPE, dev)
    if Tk != T:
        raise ValueError("k_rope must have the rows of latent")
    qr_ptr = q_ptr = q_row = q_head = hq = 0
    if (q_rope is None) != (q is None):
        raise ValueError("q_rope and q belong together")
    if q_rope is not None:
        if q_rope.dtype is not torch.bfloat16:
            raise TypeError(f"q_rope must be bfloat16, got {q_rope.dtype}")
        shape, s = q_rope.shape, q_rope.stride()
        if len(shape) != 3 or shape[0] != T or shape[2] != ROPE or s[2] != 1 or q_rope.get_device() != dev:
            raise ValueError("q_rope must be [T, Hq, 64] on the cache's device, with contiguous columns")
        hq = shape[1]
        q_head = s[1] if hq > 1 else ROPE
        q_row = s[0] if T > 1 else hq * ROPE
        _check_like(q, (T, hq, cs.rank + ROPE), torch.bfloat16, dev, "q")
        qr_ptr, q_ptr = q_rope.data_ptr(), q.data_ptr()
    rope_ptr = rope_len = 0
    if rope is not None:
        if (rope.dtype is not torch.float32 or rope.dim() != 2 or rope.shape[1] != ROPE or rope.get_device() != dev
                or not rope.is_contiguous()):
            raise ValueError("rope must be a contiguous fp32 [positions, 64] tensor on the cache's device")
        rope_ptr, rope_len = rope.data_ptr(), rope.shape[0]
    _call(_lib.load().fattn_latent_append, dev, ctypes.byref(cs), latent.data_ptr(), latent_row, k_rope.data_ptr(), k_row,
          qr_ptr, q_row, q_head, q_ptr, hq, rope_ptr, rope_len, 1 if interleaved else 0, page_table.data_ptr(),
          q_start.data_ptr(), kv_len.data_ptr(), T, B, max_pages)
    return q


@functools.lru_cache(maxsize=1024)
def fattn_latent_fwd_workspace_bytes(T: int, B: int, Hq: int, rank: int) -> int:
    return int(_lib.load().fattn_latent_fwd_workspace_bytes(T, B, Hq, rank))


def fattn_latent_fwd(q, cache: LatentCache, page_table, q_start, kv_len, scale: float, causal: bool = True, out=None,
                     lse=None, workspace=None):
    """Attention of bf16 [T, Hq, rank + 64] rows (absorbed queries and their
    rotated parts) over their sequences' cached tokens; returns (O bf16 [T, Hq,
    rank], L fp32 [T, Hq]).  ``scale`` is that of the heads before their
    projection was absorbed, so it has no default.  One layout serves the whole
    batch, chosen by its average sequence and, for many rows, the table's room:
    pieces of prompts and many single tokens are faster in two calls than in one."""
    cs, dev = _check_latent(cache)
    B, max_pages = _check_batch(page_table, q_start, kv_len, dev)
    if q.dtype is not torch.bfloat16:
        raise TypeError(f"q must be bfloat16, got {q.dtype}")
    shape, rank = q.shape, cs.rank
    if len(shape) != 3 or shape[2] != rank + ROPE or q.get_device() != dev or not q.is_contiguous():
        raise ValueError("q must be a contiguous [T, Hq, rank + 64] tensor on the cache's device")
    T, heads, _ = shape
    device = q.device
    if out is None:
        out = torch.empty((T, heads, rank), dtype=torch.bfloat16, device=device)
    else:
        _check_like(out, (T, heads, rank), torch.bfloat16, dev, "out")
    if lse is None:
        lse = torch.empty((T, heads), dtype=torch.float32, device=device)
    else:
        _check_like(lse, (T, heads), torch.float32, dev, "lse")
    need = fattn_latent_fwd_workspace_bytes(T, B, heads, rank)
    scratch = 0
    if workspace is None and need and _raw_alloc and _raw_free and _current_device() == dev:
        # as in fattn_cache_fwd: a block that the stream's next calls may have
        scratch = ws_ptr = _raw_alloc(need, _raw_stream(dev))
    else:
        ws = _workspace(workspace, need, device, dev)
        ws_ptr, need = ws.data_ptr(), ws.numel()
    try:
        _call(_lib.load().fattn_latent_fwd, dev, ctypes.byref(cs), q.data_ptr(), out.data_ptr(), lse.data_ptr(),
              page_table.data_ptr(), q_start.data_ptr(), kv_len.data_ptr(), ws_ptr, need, T, B, heads, max_pages,
              1 if causal else 0, float(scale))
    finally:
        if scratch:
            _raw_free(scratch)
    return out, lse
