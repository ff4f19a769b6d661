"""Rotary positions of queries, keys and their gradients, with the C ABI's names."""

from __future__ import annotations

import torch

from . import _lib
from .cache import _call


def _view(t, name, d, dev):
    """Strides of a [B, H, N, d] tensor, or of [T, H, d] rows as [1, H, T, d]; 0 for
    dimensions of one, whose strides may be any number."""
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the table's device")
    shape, s = t.shape, t.stride()
    if shape[-1] != d or (d > 1 and s[-1] != 1):
        raise ValueError(f"the columns of {name} must be contiguous")
    s = [x if n > 1 else 0 for n, x in zip(shape, s)]
    return (0, s[1], s[0]) if len(s) == 3 else s[:3]


def _rotate(name, x, rope, positions, interleaved, transposed, out):
    dev = rope.get_device()
    if dev < 0:
        raise ValueError("libfattn works on CUDA tensors; move the table to the GPU first")
    if rope.dtype is not torch.float32 or rope.dim() != 2 or not rope.is_contiguous():
        raise ValueError("rope must be a contiguous fp32 [positions, rope_dim] tensor")
    shape = x.shape
    if len(shape) == 4:
        B, H, N, d = shape
    elif len(shape) == 3:
        B, (N, H, d) = 1, shape
    else:
        raise ValueError(f"{name} must be [B, H, N, d] or rows [T, H, d]")
    xs = _view(x, name, d, dev)
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=x.device)
    elif out.shape != shape:
        raise ValueError(f"out must have the shape of {name}")
    ys = _view(out, "out", d, dev)
    pos, pos_stride = 0, 0
    if positions is not None:
        pshape = positions.shape
        if positions.dtype is not torch.int32 or positions.get_device() != dev or not positions.is_contiguous():
            raise ValueError("positions must be a contiguous int32 tensor on the table's device")
        if len(pshape) == 2 and len(shape) == 4:
            pos_stride = N
            good = pshape == (B, N)
        else:
            good = pshape == (N,)
        if not good:
            raise ValueError("positions must be [N] or [B, N], or [T] for rows")
        pos = positions.data_ptr()
    rope_len, rope_dim = rope.shape
    if B * H * N == 0:
        return out
    _call(_lib.load().fattn_rope, dev, x.data_ptr(), *xs, out.data_ptr(), *ys, rope.data_ptr(), rope_len, rope_dim,
          1 if interleaved else 0, 1 if transposed else 0, pos, pos_stride, B, H, N, d)
    return out


def fattn_rope(x, rope, positions=None, interleaved: bool = False, out=None):
    """Rotate the pairs of x's first rope_dim columns by their rows' positions
    (``rope`` from fattn_rope_table, fp32 [positions, rope_dim]).  ``x`` is bf16
    [B, H, N, d] or rows [T, H, d] and may be strided, so a slice of the columns
    is rotated as a view; ``positions`` is int32 [N], [B, N] or [T], by default
    0 .. N-1.  ``out`` may be ``x``.  Rows of a position outside the table are not
    written."""
    return _rotate("x", x, rope, positions, interleaved, False, out)


def fattn_rope_bwd(dy, rope, positions=None, interleaved: bool = False, out=None):
    """The gradient of fattn_rope's input for its output's: dx = R^T dy, the
    rotation by the negated angles (with the table's magnitude)."""
    return _rotate("dy", dy, rope, positions, interleaved, True, out)
