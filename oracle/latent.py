"""Paged latent cache: appending and attention over it.

TEST INFRASTRUCTURE ONLY (see the package docstring): it shares no code with
the CUDA library.  The pages do not treat such a cache; these are the
definitions that include/fattn.h states.  Data is float32 [pages, page, rank +
64] of bf16 values.
"""

from __future__ import annotations

import numpy as np

from .rope import rotate_fp32

ROPE = 64


def _bf16(x):
    """fp32 rounded to bf16 (nearest even), as fp32."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16 << 16).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(x), np.float32(np.nan), r)


def append(data, latent, k_rope, table, q_start, kv_len, rope=None, interleaved=False, q_rope=None, q=None):
    """Updates ``data`` and ``q`` in place."""
    page, rank = data.shape[1], latent.shape[1]
    for b in range(len(kv_len)):
        r0, n = int(q_start[b]), int(q_start[b + 1] - q_start[b])
        for i in range(n):
            t = int(kv_len[b]) - n + i
            row = r0 + i
            key, ang = k_rope[row], None if rope is None else rope[t]
            if rope is not None:
                key = _bf16(rotate_fp32(key, ang, interleaved))
            new = np.concatenate([latent[row], key])
            if not np.isfinite(new).all():
                new[:rank], new[rank:] = 0.0, np.nan
            data[int(table[b, t // page]), t % page] = new
            if q is not None:
                q[row, :, rank:] = q_rope[row] if rope is None else _bf16(rotate_fp32(q_rope[row], ang, interleaved))


def tokens(data, table_row, n):
    """The first n cached rows of a sequence, float64; NaN rows where the table
    names no page."""
    page = data.shape[1]
    out = np.full((n, data.shape[2]), np.nan)
    for p in range(-(-n // page)):
        pid = int(table_row[p])
        if 0 <= pid < data.shape[0]:
            m = min(page, n - p * page)
            out[p * page:p * page + m] = data[pid, :m]
    return out


def attend(q, data, rank, table, q_start, kv_len, causal, scale):
    """(O, L, A, D): outputs, log sums, the probabilities' sum of |values|, and
    the largest scale * sum |q k| of a row; NaN in L for rows of no sequence.
    Tokens on pages that do not exist count as absent."""
    T, heads, _ = q.shape
    O, A = np.zeros((T, heads, rank)), np.zeros((T, heads, rank))
    L, D = np.full((T, heads), np.nan), np.zeros((T, heads))
    for b in range(len(kv_len)):
        r0, n, t = int(q_start[b]), int(q_start[b + 1] - q_start[b]), int(kv_len[b])
        if n == 0:
            continue
        k = tokens(data, table[b], t)
        there = np.ones(t, bool)
        for p in range(-(-t // data.shape[1])):
            if not 0 <= int(table[b, p]) < data.shape[0]:
                there[p * data.shape[1]:(p + 1) * data.shape[1]] = False
        for i in range(n):
            see = max(0, min(t, t - n + i + 1)) if causal else t
            kk = k[:see][there[:see]]
            if not len(kk):
                L[r0 + i] = -np.inf
                continue
            x = scale * (q[r0 + i].astype(np.float64) @ kk.T)
            m = x.max(axis=1, keepdims=True)
            p = np.exp(x - m)
            l = p.sum(axis=1, keepdims=True)
            O[r0 + i], A[r0 + i] = (p / l) @ kk[:, :rank], (p / l) @ np.abs(kk[:, :rank])
            L[r0 + i] = (m + np.log(l))[:, 0]
            D[r0 + i] = (scale * (np.abs(q[r0 + i].astype(np.float64)) @ np.abs(kk).T)).max(axis=1)
    return O, L, A, D
