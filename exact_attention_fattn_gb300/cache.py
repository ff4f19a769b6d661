"""Python entry points of the paged 8-bit cache, with the C ABI's names.

As in attention.py, PyTorch provides device memory and streams only: the
functions check what the host can see, allocate outputs and workspaces, and
hand raw pointers and the current CUDA stream to the library.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import _lib
from .attention import _check_out, _stream_ptr, default_scale

PAGE_SIZES = (32, 64, 128)


class Fp8Cache(NamedTuple):
    """A caller-owned cache: e4m3 codes, one power-of-two scale per page and
    kv head, and (for fattn_cache_select) per-page bounds of the keys."""

    k: torch.Tensor                 # uint8 [pages, Hkv, page, d]
    v: torch.Tensor                 # uint8 [pages, Hkv, page, d]
    k_scale: torch.Tensor           # fp32 [pages, Hkv]
    v_scale: torch.Tensor           # fp32 [pages, Hkv]
    k_bounds: Optional[torch.Tensor] = None   # int8 [pages, Hkv, 2, d]


def fattn_cache_alloc(pages: int, kv_heads: int, d: int, page: int = 64, device="cuda",
                      bounds: bool = False) -> Fp8Cache:
    """An empty cache of ``pages`` pages of ``page`` tokens (codes zero, scales 1)."""
    if pages < 1 or kv_heads < 1 or page not in PAGE_SIZES or d not in (64, 128):
        raise ValueError("need pages, kv_heads >= 1, page in (32, 64, 128) and d in (64, 128)")
    k, v = (torch.zeros((pages, kv_heads, page, d), dtype=torch.uint8, device=device)
            for _ in range(2))
    ks, vs = (torch.ones((pages, kv_heads), dtype=torch.float32, device=device) for _ in range(2))
    b = (torch.zeros((pages, kv_heads, 2, d), dtype=torch.int8, device=device) if bounds else None)
    return Fp8Cache(k, v, ks, vs, b)


def fattn_rope_table(positions: int, rope_dim: int, theta: float = 10000.0,
                     device="cuda") -> torch.Tensor:
    """fp32 [positions, rope_dim]: the cosines, then the sines, of the angles
    p * theta**(-2 i / rope_dim); taken in 64 bits, for far positions."""
    if positions < 1 or rope_dim < 16 or rope_dim % 16:
        raise ValueError("rope_dim must be a multiple of 16, and there must be a position")
    inv = theta ** (-torch.arange(0, rope_dim, 2, dtype=torch.float64, device=device) / rope_dim)
    ang = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], dim=1).float()


def _check_cache(c: Fp8Cache) -> _lib.CacheStruct:
    k, v = c.k, c.v
    if not k.is_cuda:
        raise ValueError("libfattn works on CUDA tensors; move the cache to the GPU first")
    if k.dim() != 4 or v.shape != k.shape:
        raise ValueError("cache k and v must share one [pages, Hkv, page, d] shape")
    pages, heads, page, d = k.shape
    if k.dtype != torch.uint8 or v.dtype != torch.uint8:
        raise TypeError("cache k and v must be uint8 (e4m3 codes)")
    stride = k.stride(0) if pages > 1 else heads * page * d
    for t in (k, v):
        if t.stride()[1:] != (page * d, d, 1) or (pages > 1 and t.stride(0) != stride):
            raise ValueError("cache pages must be contiguous and equally spaced in k and v")
    dev = k.device
    for t, name in ((c.k_scale, "k_scale"), (c.v_scale, "v_scale")):
        _check_out(t, (pages, heads), torch.float32, dev, name)
    if v.device != dev:
        raise ValueError("the cache must be on one device")
    bounds = 0
    if c.k_bounds is not None:
        bounds = _check_out(c.k_bounds, (pages, heads, 2, d), torch.int8, dev, "k_bounds").data_ptr()
    return _lib.CacheStruct(k.data_ptr(), v.data_ptr(), c.k_scale.data_ptr(), c.v_scale.data_ptr(),
                            bounds, stride, pages, heads, page, d)


def _check_batch(page_table, q_start, kv_len, dev):
    for t, name in ((page_table, "page_table"), (q_start, "q_start"), (kv_len, "kv_len")):
        if t.dtype != torch.int32 or t.device != dev or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 tensor on {dev}")
    B = kv_len.numel()
    if (page_table.dim() != 2 or page_table.shape[0] != B or kv_len.dim() != 1
            or q_start.shape != (B + 1,)):
        raise ValueError("need page_table [B, max_pages], q_start [B + 1] and kv_len [B]")
    return B, page_table.shape[1]


def _check_rows(t, name, T, heads, d, dev):
    """bf16 [T, heads, d] whose rows may lie apart; their distance in elements."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    if t.dim() != 3 or t.shape[2] != d or (T is not None and t.shape[0] != T) or (
            heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be [T, heads, d] with the call's T, heads and d = {d}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}")
    row = t.shape[1] * d
    if t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != d):
        raise ValueError(f"the heads of a row of {name} must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else row


def fattn_cache_append(k_new, v_new, cache: Fp8Cache, page_table, q_start, kv_len, rope=None, q=None,
                       interleaved: bool = False, q_out=None):
    """Append new tokens (bf16 [T, Hkv, d]) to their sequences' pages, keys
    rotated by ``rope`` (fattn_rope_table); returns the rotated queries (bf16
    [T, Hq, d]) when ``q`` is given, else None.  q_start [B + 1], kv_len [B]
    (the new tokens included) and page_table [B, max_pages] are int32 CUDA
    tensors; rows from q_start[B] on are left alone."""
    cs = _check_cache(cache)
    dev = cache.k.device
    B, max_pages = _check_batch(page_table, q_start, kv_len, dev)
    T = k_new.shape[0] if k_new.dim() == 3 else None
    k_row = _check_rows(k_new, "k_new", T, cs.Hkv, cs.d, dev)
    v_row = _check_rows(v_new, "v_new", T, cs.Hkv, cs.d, dev)
    q_ptr = out_ptr = q_row = heads = 0
    if q is not None:
        heads = q.shape[1] if q.dim() == 3 else 0
        q_row = _check_rows(q, "q", T, None, cs.d, dev)
        q_out = (torch.empty(q.shape, dtype=q.dtype, device=dev) if q_out is None
                 else _check_out(q_out, q.shape, q.dtype, dev, "q_out"))
        q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    rope_ptr = rope_len = rope_dim = 0
    if rope is not None:
        if rope.dtype != torch.float32 or rope.dim() != 2 or rope.device != dev or not rope.is_contiguous():
            raise ValueError(f"rope must be a contiguous fp32 [positions, rope_dim] tensor on {dev}")
        rope_ptr, (rope_len, rope_dim) = rope.data_ptr(), rope.shape
    with torch.cuda.device(dev):
        rc = _lib.load().fattn_cache_append(
            ctypes.byref(cs), k_new.data_ptr(), k_row, v_new.data_ptr(), v_row, q_ptr, q_row, out_ptr,
            heads, rope_ptr, rope_len, rope_dim, int(bool(interleaved)), page_table.data_ptr(),
            q_start.data_ptr(), kv_len.data_ptr(), T, B, max_pages, _stream_ptr(dev))
    _lib.check("fattn_cache_append", rc)
    return q_out


def _check_workspace(ws, need, dev):
    if need == 0:
        raise ValueError("unsupported sizes")
    if ws is None:
        return torch.empty(need, dtype=torch.uint8, device=dev)
    if ws.dtype != torch.uint8 or ws.device != dev or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the inputs' device")
    return ws   # its size is checked by the library


def fattn_cache_fwd_workspace_bytes(T: int, B: int, Hq: int, Hkv: int, d: int,
                                    n_selected: int = 0) -> int:
    return int(_lib.load().fattn_cache_fwd_workspace_bytes(T, B, Hq, Hkv, d, n_selected))


def fattn_cache_fwd(q, cache: Fp8Cache, page_table, q_start, kv_len, causal: bool = True,
                    scale: float | None = None, selected=None, out=None, lse=None, workspace=None):
    """Attention of bf16 [T, Hq, d] rows over their sequences' cached tokens;
    returns (O bf16 [T, Hq, d], L fp32 [T, Hq]).  With ``selected`` (int32
    [T, Hkv, n], from fattn_cache_select) a row attends to those pages only."""
    cs = _check_cache(cache)
    dev = cache.k.device
    B, max_pages = _check_batch(page_table, q_start, kv_len, dev)
    q_row = _check_rows(q, "q", None, None, cs.d, dev)
    T, heads, d = q.shape
    scale = default_scale(d) if scale is None else float(scale)
    n_sel = sel_ptr = 0
    if selected is not None:
        if (selected.dtype != torch.int32 or selected.dim() != 3 or selected.shape[:2] != (T, cs.Hkv)
                or selected.shape[2] < 1 or selected.device != dev or not selected.is_contiguous()):
            raise ValueError(f"selected must be a contiguous int32 [T, Hkv, n] tensor on {dev}")
        n_sel, sel_ptr = selected.shape[2], selected.data_ptr()
    o = (torch.empty((T, heads, d), dtype=q.dtype, device=dev) if out is None
         else _check_out(out, (T, heads, d), q.dtype, dev, "out"))
    l = (torch.empty((T, heads), dtype=torch.float32, device=dev) if lse is None
         else _check_out(lse, (T, heads), torch.float32, dev, "lse"))
    lib = _lib.load()
    ws = _check_workspace(workspace, lib.fattn_cache_fwd_workspace_bytes(T, B, heads, cs.Hkv, d, n_sel),
                          dev)
    with torch.cuda.device(dev):
        rc = lib.fattn_cache_fwd(ctypes.byref(cs), q.data_ptr(), q_row, o.data_ptr(), l.data_ptr(),
                                 page_table.data_ptr(), q_start.data_ptr(), kv_len.data_ptr(), sel_ptr,
                                 n_sel, ws.data_ptr(), ws.numel(), T, B, heads, max_pages,
                                 int(bool(causal)), scale, _stream_ptr(dev))
    _lib.check("fattn_cache_fwd", rc)
    return o, l


def fattn_cache_select_workspace_bytes(T: int, Hkv: int, max_pages: int) -> int:
    return int(_lib.load().fattn_cache_select_workspace_bytes(T, Hkv, max_pages))


def fattn_cache_select(q, cache: Fp8Cache, page_table, q_start, kv_len, n_selected: int,
                       n_first: int = 0, n_recent: int = 1, out=None, workspace=None):
    """The ``n_selected`` pages of each row's sequence that its queries may
    score highest on, per kv head: int32 [T, Hkv, n_selected], ascending, -1
    behind the last.  The first ``n_first`` and last ``n_recent`` are always
    among them.  The cache needs its bounds."""
    cs = _check_cache(cache)
    dev = cache.k.device
    if cache.k_bounds is None:
        raise ValueError("the cache was made without bounds")
    B, max_pages = _check_batch(page_table, q_start, kv_len, dev)
    q_row = _check_rows(q, "q", None, None, cs.d, dev)
    T, heads, _ = q.shape
    sel = (torch.empty((T, cs.Hkv, n_selected), dtype=torch.int32, device=dev) if out is None
           else _check_out(out, (T, cs.Hkv, n_selected), torch.int32, dev, "out"))
    lib = _lib.load()
    ws = _check_workspace(workspace, lib.fattn_cache_select_workspace_bytes(T, cs.Hkv, max_pages), dev)
    with torch.cuda.device(dev):
        rc = lib.fattn_cache_select(ctypes.byref(cs), q.data_ptr(), q_row, page_table.data_ptr(),
                                    q_start.data_ptr(), kv_len.data_ptr(), sel.data_ptr(), n_selected,
                                    n_first, n_recent, ws.data_ptr(), ws.numel(), T, B, heads, max_pages,
                                    _stream_ptr(dev))
    _lib.check("fattn_cache_select", rc)
    return sel
