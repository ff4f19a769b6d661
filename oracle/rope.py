"""Rotary positions in plain NumPy.

TEST INFRASTRUCTURE ONLY (see the package docstring): it shares no code with
the CUDA library.  The pages do not treat rotations; these are the definitions
that include/fattn.h states.
"""

from __future__ import annotations

import numpy as np

F = np.float32


def _pairs(rope_dim, interleaved):
    h = rope_dim // 2
    return (np.arange(0, rope_dim, 2), np.arange(1, rope_dim, 2)) if interleaved else (np.arange(h), np.arange(h, rope_dim))


def rotate_fp32(x, table, interleaved=False, transposed=False):
    """x fp32 [..., d], table fp32 [..., rope_dim] (cosines, then sines), of
    shapes that broadcast without their last: every product and sum rounded."""
    h = table.shape[-1] // 2
    c, s = table[..., :h].astype(F), table[..., h:].astype(F)
    if transposed:
        s = -s
    ia, ib = _pairs(2 * h, interleaved)
    y = x.astype(F).copy()
    a, b = y[..., ia].copy(), y[..., ib].copy()
    with np.errstate(invalid="ignore", over="ignore"):
        y[..., ia] = (a * c).astype(F) - (b * s).astype(F)
        y[..., ib] = (b * c).astype(F) + (a * s).astype(F)
    return y


def rotate(x, angles, interleaved=False, magnitude=1.0):
    """The rotation itself in 64 bits: x [..., d], angles [..., rope_dim / 2]."""
    x = np.asarray(x, dtype=np.float64)
    ia, ib = _pairs(2 * angles.shape[-1], interleaved)
    y = x.copy()
    z = (x[..., ia] + 1j * x[..., ib]) * (magnitude * np.exp(1j * angles))
    y[..., ia], y[..., ib] = z.real, z.imag
    return y


def frequencies(rope_dim, theta=10000.0, factor=1.0, original=0, ramp=(1.0, 32.0)):
    """Angle per position of each pair."""
    inv = float(theta) ** (-np.arange(0, rope_dim, 2, dtype=np.float64) / rope_dim)
    if not original:
        return inv / factor
    out = np.empty_like(inv)
    for i, f in enumerate(inv):
        turns = original * f / (2 * np.pi)
        keep = min(1.0, max(0.0, (turns - ramp[0]) / (ramp[1] - ramp[0])))
        out[i] = keep * f + (1.0 - keep) * f / factor
    return out
