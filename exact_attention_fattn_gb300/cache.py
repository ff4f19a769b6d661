"""Python entry points of the paged 8-bit cache, with the C ABI's names.

As in attention.py, PyTorch provides device memory and streams only: the
functions check what the host can see, allocate outputs and workspaces, and
hand raw pointers and the current CUDA stream to the library.
"""

from __future__ import annotations

import ctypes
import functools
import math
from typing import NamedTuple, Optional

import torch

from . import _lib
from .attention import default_scale

PAGE_SIZES = (32, 64, 128)
MAX_KV_HEADS = 1024


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
    if pages < 1 or not 1 <= kv_heads <= MAX_KV_HEADS or page not in PAGE_SIZES or d not in (64, 128):
        raise ValueError(f"need pages >= 1, kv_heads from 1 to {MAX_KV_HEADS}, page in (32, 64, 128) and d in (64, 128)")
    k, v = (torch.zeros((pages, kv_heads, page, d), dtype=torch.uint8, device=device)
            for _ in range(2))
    ks, vs = (torch.ones((pages, kv_heads), dtype=torch.float32, device=device) for _ in range(2))
    b = (torch.zeros((pages, kv_heads, 2, d), dtype=torch.int8, device=device) if bounds else None)
    return Fp8Cache(k, v, ks, vs, b)


def fattn_rope_table(positions: int, rope_dim: int, theta: float = 10000.0, device="cuda", factor: float = 1.0,
                     original: int = 0, ramp: tuple = (1.0, 32.0), magnitude: float | None = None) -> torch.Tensor:
    """fp32 [positions, rope_dim]: the cosines, then the sines, of the angles
    p * theta**(-2 i / rope_dim); taken in 64 bits, for far positions.

    For contexts ``factor`` times as long as the model was trained on, angles
    are divided by the factor: all of them (``original`` 0), or, with
    ``original`` the trained length, those that turn less than ramp[0] times in
    it, while those that turn ramp[1] times or more stay and those between go
    over linearly in their turns (a model whose angles go over in another way
    brings a table of its own: any fp32 one is taken); the table is then multiplied by ``magnitude`` (by default
    0.1 ln(factor) + 1), which scales the scores by its square."""
    if positions < 1 or rope_dim < 16 or rope_dim % 16:
        raise ValueError("rope_dim must be a multiple of 16, and there must be a position")
    if not (factor >= 1.0 and math.isfinite(factor)) or original < 0 or not 0 <= ramp[0] < ramp[1]:
        raise ValueError("need a factor of 1 or more, original >= 0 and 0 <= ramp[0] < ramp[1]")
    inv = theta ** (-torch.arange(0, rope_dim, 2, dtype=torch.float64, device=device) / rope_dim)
    if original:
        keep = ((original * inv / (2 * math.pi) - ramp[0]) / (ramp[1] - ramp[0])).clamp(0.0, 1.0)
        inv = inv * (keep + (1.0 - keep) / factor)
        if magnitude is None:
            magnitude = 0.1 * math.log(factor) + 1.0
    else:
        inv = inv / factor
    ang = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * inv
    return (torch.cat([ang.cos(), ang.sin()], dim=1) * (1.0 if magnitude is None else magnitude)).float()


# The functions below run once per layer and token, where a call's latency is
# mostly the host's: each attribute of a tensor is read once, devices are
# compared by index, and the scale, the stream and the current device come
# without a tensor or a context manager.  On GB300's host a call of
# fattn_cache_fwd took 44.7 us before and 22 us so, 6 of them for the library.

_SCALES = {d: default_scale(d) for d in (64, 128)}


def _check_cache(c: Fp8Cache):
    """The C ABI's description of the cache, its device index and device."""
    k, v, ks, vs, kb = c
    shape, dev = k.shape, k.get_device()
    if dev < 0:
        raise ValueError("libfattn works on CUDA tensors; move the cache to the GPU first")
    if len(shape) != 4 or v.shape != shape:
        raise ValueError("cache k and v must share one [pages, Hkv, page, d] shape")
    if k.dtype is not torch.uint8 or v.dtype is not torch.uint8:
        raise TypeError("cache k and v must be uint8 (e4m3 codes)")
    pages, heads, page, d = shape
    s = k.stride()
    if s[3] != 1 or s[2] != d or s[1] != page * d or v.stride() != s:
        raise ValueError("cache pages must be contiguous and equally spaced in k and v")
    stride = s[0] if pages > 1 else heads * page * d
    sshape = shape[:2]
    if (ks.shape != sshape or vs.shape != sshape or ks.dtype is not torch.float32
            or vs.dtype is not torch.float32 or not ks.is_contiguous() or not vs.is_contiguous()):
        raise ValueError("k_scale and v_scale must be contiguous fp32 [pages, Hkv] tensors")
    if v.get_device() != dev or ks.get_device() != dev or vs.get_device() != dev:
        raise ValueError("the cache must be on one device")
    bounds = 0
    if kb is not None:
        if (kb.shape != (pages, heads, 2, d) or kb.dtype is not torch.int8 or not kb.is_contiguous()
                or kb.get_device() != dev):
            raise ValueError("k_bounds must be a contiguous int8 [pages, Hkv, 2, d] tensor on the cache's device")
        bounds = kb.data_ptr()
    return _lib.CacheStruct(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), bounds, stride,
                            pages, heads, page, d), dev


def _check_batch(page_table, q_start, kv_len, dev):
    for t in (page_table, q_start, kv_len):
        if t.dtype is not torch.int32 or t.get_device() != dev or not t.is_contiguous():
            raise ValueError("page_table, q_start and kv_len must be contiguous int32 tensors on the "
                             "cache's device")
    n, B1, tshape = kv_len.shape, q_start.shape, page_table.shape
    if len(n) != 1 or len(tshape) != 2 or tshape[0] != n[0] or len(B1) != 1 or B1[0] != n[0] + 1:
        raise ValueError("need page_table [B, max_pages], q_start [B + 1] and kv_len [B]")
    return tshape


def _check_rows(t, name, d, dev):
    """bf16 [T, heads, d] whose rows may lie apart: (T, heads, their distance
    in elements)."""
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[2] != d:
        raise ValueError(f"{name} must be [T, heads, d] with d = {d}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the cache's device")
    T, heads, _ = shape
    s = t.stride()
    if s[2] != 1 or (heads > 1 and s[1] != d):
        raise ValueError(f"the heads of a row of {name} must be contiguous")
    return T, heads, s[0] if T > 1 else heads * d


def _check_like(t, shape, dtype, dev, name):
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on the "
                         "cache's device")
    return t


def _public_stream(dev: int) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


# torch's own shortcuts where this torch has them (one without CUDA has none, and
# they carry no promise), else what is public.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _public_stream)
_raw_alloc = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc", None)
_raw_free = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_delete", None)


def _call(fn, dev, *args):
    """fn(*args, stream) on device dev, with its current stream."""
    if _current_device() == dev:
        rc = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(dev))
    if rc != _lib.FATTN_OK:
        _lib.check(fn.__name__, rc)


def fattn_cache_append(k_new, v_new, cache: Fp8Cache, page_table, q_start, kv_len, rope=None, q=None,
                       interleaved: bool = False, q_out=None):
    """Append new tokens (bf16 [T, Hkv, d]) to their sequences' pages, keys
    rotated by ``rope`` (fattn_rope_table); returns the rotated queries (bf16
    [T, Hq, d]) when ``q`` is given, else None.  q_start [B + 1], kv_len [B]
    (the new tokens included) and page_table [B, max_pages] are int32 CUDA
    tensors; rows from q_start[B] on are left alone."""
    cs, dev = _check_cache(cache)
    B, max_pages = _check_batch(page_table, q_start, kv_len, dev)
    T, heads, k_row = _check_rows(k_new, "k_new", cs.d, dev)
    Tv, heads_v, v_row = _check_rows(v_new, "v_new", cs.d, dev)
    if heads != cs.Hkv or heads_v != heads or Tv != T:
        raise ValueError("k_new and v_new must be [T, Hkv, d] with the cache's Hkv")
    q_ptr = out_ptr = q_row = hq = 0
    if q is not None:
        Tq, hq, q_row = _check_rows(q, "q", cs.d, dev)
        if Tq != T:
            raise ValueError("q must have the rows of k_new")
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        else:
            _check_like(q_out, q.shape, torch.bfloat16, dev, "q_out")
        q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    rope_ptr = rope_len = rope_dim = 0
    if rope is not None:
        if rope.dtype is not torch.float32 or rope.dim() != 2 or rope.get_device() != dev or not rope.is_contiguous():
            raise ValueError("rope must be a contiguous fp32 [positions, rope_dim] tensor on the cache's device")
        rope_ptr, (rope_len, rope_dim) = rope.data_ptr(), rope.shape
    _call(_lib.load().fattn_cache_append, dev, ctypes.byref(cs), k_new.data_ptr(), k_row, v_new.data_ptr(),
          v_row, q_ptr, q_row, out_ptr, hq, rope_ptr, rope_len, rope_dim, 1 if interleaved else 0,
          page_table.data_ptr(), q_start.data_ptr(), kv_len.data_ptr(), T, B, max_pages)
    return q_out


def _workspace(ws, need, device, dev):
    if need == 0:
        raise ValueError("unsupported sizes")
    if ws is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if ws.dtype is not torch.uint8 or ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the inputs' device")
    return ws   # its size is checked by the library


@functools.lru_cache(maxsize=1024)
def fattn_cache_fwd_workspace_bytes(T: int, B: int, Hq: int, Hkv: int, d: int,
                                    n_selected: int = 0) -> int:
    return int(_lib.load().fattn_cache_fwd_workspace_bytes(T, B, Hq, Hkv, d, n_selected))


def fattn_cache_fwd(q, cache: Fp8Cache, page_table, q_start, kv_len, causal: bool = True,
                    scale: float | None = None, selected=None, out=None, lse=None, workspace=None):
    """Attention of bf16 [T, Hq, d] rows over their sequences' cached tokens;
    returns (O bf16 [T, Hq, d], L fp32 [T, Hq]).  With ``selected`` (int32
    [T, Hkv, n], from fattn_cache_select) a row attends to those pages only.
    One kernel serves the whole batch, chosen by its average sequence: pieces of
    prompts and many single tokens are faster in two calls than in one."""
    cs, dev = _check_cache(cache)
    B, max_pages = _check_batch(page_table, q_start, kv_len, dev)
    d = cs.d
    T, heads, q_row = _check_rows(q, "q", d, dev)
    n_sel = sel_ptr = 0
    if selected is not None:
        n_sel = selected.shape[-1]
        if n_sel < 1:
            raise ValueError("selected must name at least one page a row")
        _check_like(selected, (T, cs.Hkv, n_sel), torch.int32, dev, "selected")
        sel_ptr = selected.data_ptr()
    device = q.device
    if out is None:
        out = torch.empty((T, heads, d), dtype=torch.bfloat16, device=device)
    else:
        _check_like(out, (T, heads, d), torch.bfloat16, dev, "out")
    if lse is None:
        lse = torch.empty((T, heads), dtype=torch.float32, device=device)
    else:
        _check_like(lse, (T, heads), torch.float32, dev, "lse")
    need = fattn_cache_fwd_workspace_bytes(T, B, heads, cs.Hkv, d, n_sel)
    scratch = 0
    if workspace is None and need and _raw_alloc and _raw_free and _current_device() == dev:
        # a block of the allocator that the stream's next calls may have, without a tensor around it
        scratch = ws_ptr = _raw_alloc(need, _raw_stream(dev))
    else:
        ws = _workspace(workspace, need, device, dev)
        ws_ptr, need = ws.data_ptr(), ws.numel()
    try:
        _call(_lib.load().fattn_cache_fwd, dev, ctypes.byref(cs), q.data_ptr(), q_row, out.data_ptr(), lse.data_ptr(),
              page_table.data_ptr(), q_start.data_ptr(), kv_len.data_ptr(), sel_ptr, n_sel, ws_ptr, need, T, B,
              heads, max_pages, 1 if causal else 0, (_SCALES.get(d, 1.0) if scale is None else float(scale)))
    finally:
        if scratch:
            _raw_free(scratch)
    return out, lse


@functools.lru_cache(maxsize=1024)
def fattn_cache_select_workspace_bytes(T: int, Hkv: int, max_pages: int) -> int:
    return int(_lib.load().fattn_cache_select_workspace_bytes(T, Hkv, max_pages))


def fattn_cache_select(q, cache: Fp8Cache, page_table, q_start, kv_len, n_selected: int,
                       n_first: int = 0, n_recent: int = 1, out=None, workspace=None):
    """The ``n_selected`` pages of each row's sequence that its queries may
    score highest on, per kv head: int32 [T, Hkv, n_selected], ascending, -1
    behind the last.  The first ``n_first`` and last ``n_recent`` are always
    among them.  The cache needs its bounds."""
    cs, dev = _check_cache(cache)
    if cache.k_bounds is None:
        raise ValueError("the cache was made without bounds")
    B, max_pages = _check_batch(page_table, q_start, kv_len, dev)
    T, heads, q_row = _check_rows(q, "q", cs.d, dev)
    if out is None:
        if n_selected < 1:
            raise ValueError("n_selected must be at least 1")
        out = torch.empty((T, cs.Hkv, n_selected), dtype=torch.int32, device=q.device)
    else:
        _check_like(out, (T, cs.Hkv, n_selected), torch.int32, dev, "out")
    need = fattn_cache_select_workspace_bytes(T, cs.Hkv, max_pages)
    ws_ptr = ws_bytes = 0
    if workspace is not None or need != 256:   # 256: the scores stay on chip
        ws = _workspace(workspace, need, q.device, dev)
        ws_ptr, ws_bytes = ws.data_ptr(), ws.numel()
    _call(_lib.load().fattn_cache_select, dev, ctypes.byref(cs), q.data_ptr(), q_row, page_table.data_ptr(),
          q_start.data_ptr(), kv_len.data_ptr(), out.data_ptr(), n_selected, n_first, n_recent,
          ws_ptr, ws_bytes, T, B, heads, max_pages)
    return out
