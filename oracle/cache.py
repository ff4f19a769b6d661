"""Paged 8-bit cache: appending, attention over it, and page selection.

TEST INFRASTRUCTURE ONLY (see the package docstring): it shares no code with
the CUDA library.  The pages do not treat a cache; these are the definitions
that include/fattn.h states.

* A cache is k, v uint8 [pages, Hkv, page, d] (e4m3 codes), k_scale, v_scale
  fp32 [pages, Hkv] (powers of two) and bounds int8 [pages, Hkv, 2, d].
* What decides a code or a choice (the rotation, the scaling, the query's
  rounding to whole numbers) is taken in fp32 step by step, because its
  roundings show; attention is plain fp64.
"""

from __future__ import annotations

import numpy as np

from .fp8 import E4M3_MAX, e4m3_decode, e4m3_encode

E_MIN, E_MAX = -48, 48
F = np.float32


def rope_rotate(x, table, interleaved):
    """x fp32 [heads, d], table fp32 [rope_dim] (cosines, then sines) of the
    row's position: every product and sum rounded to fp32."""
    if table is None:
        return x.astype(F)
    h = table.shape[0] // 2
    c, s = table[:h].astype(F), table[h:].astype(F)
    y = x.astype(F).copy()
    ia, ib = (np.arange(0, 2 * h, 2), np.arange(1, 2 * h, 2)) if interleaved else (
        np.arange(h), np.arange(h, 2 * h))
    a, b = y[:, ia].copy(), y[:, ib].copy()
    with np.errstate(invalid="ignore"):
        y[:, ia] = (a * c).astype(F) - (b * s).astype(F)
        y[:, ib] = (b * c).astype(F) + (a * s).astype(F)
    return y


def scale_exponent(amax):
    """The smallest e in [-48, 48] with amax <= 448 * 2^e."""
    for e in range(E_MIN, E_MAX + 1):
        if float(amax) <= E4M3_MAX * 2.0 ** e:
            return e
    return E_MAX


def _bound_units(values):
    t = ((values.astype(F) * F(127.0)).astype(F) / F(448.0)).astype(F)
    return np.floor(t), np.ceil(t)


def append(cache, k_new, v_new, table, q_start, kv_len, rope=None, interleaved=False, q=None):
    """Updates ``cache`` (dict of arrays) in place; k_new, v_new fp32 [T, Hkv, d];
    returns the rotated queries (fp32, not yet rounded to bf16) or None."""
    page = cache["k"].shape[2]
    q_out = None if q is None else np.array(q, dtype=F)
    for b in range(len(kv_len)):
        r0, r1, n_kv = int(q_start[b]), int(q_start[b + 1]), int(kv_len[b])
        p0 = n_kv - (r1 - r0)
        for pg in range(p0 // page, -(-n_kv // page)) if r1 > r0 else ():
            toks = range(max(p0, pg * page), min(n_kv, (pg + 1) * page))
            pid = int(table[b, pg])
            for h in range(cache["k"].shape[1]):
                ks, vs = [], []
                for t in toks:
                    row = r0 + t - p0
                    ks.append(rope_rotate(k_new[row, h:h + 1], None if rope is None else rope[t],
                                          interleaved)[0])
                    vs.append(v_new[row, h].astype(F))
                _append_page(cache, pid, h, toks[0] % page, np.stack(ks), np.stack(vs))
        if q is not None:
            for row in range(r0, r1):
                t = p0 + row - r0
                q_out[row] = rope_rotate(q_out[row], None if rope is None else rope[t], interleaved)
    return q_out


def _append_page(cache, pid, h, first, ks, vs):
    bad = np.isnan(ks).any(axis=1) | np.isnan(vs).any(axis=1)
    codes, downs = {}, {}
    for name, x in (("k", ks), ("v", vs)):
        good = x[~bad]
        e = scale_exponent(np.abs(good).max()) if good.size else E_MIN
        old = int(np.log2(cache[name + "_scale"][pid, h])) if first else None
        if first:
            e = max(e, old)
            if e > old:
                was = cache[name][pid, h, :first]
                cache[name][pid, h, :first] = e4m3_encode(
                    (e4m3_decode(was).astype(F) * F(2.0 ** (old - e))).astype(F))
        downs[name] = F(2.0 ** (old - e)) if first else None
        cache[name + "_scale"][pid, h] = F(2.0 ** e)
        with np.errstate(invalid="ignore"):
            codes[name] = e4m3_encode((x * F(2.0 ** -e)).astype(F))
    codes["k"][bad] = 0x7F
    codes["v"][bad] = 0
    n = len(ks)
    for name in ("k", "v"):
        cache[name][pid, h, first:first + n] = codes[name]
    if cache.get("bounds") is None:
        return
    lo, hi = _bound_units(e4m3_decode(codes["k"][~bad]))
    b = cache["bounds"][pid, h].astype(F)
    if first:
        low, high = np.floor(b[0] * downs["k"]), np.ceil(b[1] * downs["k"])
        lo, hi = np.vstack([low[None], lo]), np.vstack([high[None], hi])
    cache["bounds"][pid, h] = (np.stack([lo.min(axis=0), hi.max(axis=0)]).astype(np.int8)
                               if len(lo) else 0)


def cached_values(cache, table_row, n_kv):
    """fp64 (k, v) [Hkv, n_kv, d] of one sequence."""
    page = cache["k"].shape[2]
    pids = np.asarray(table_row[:-(-n_kv // page)], dtype=np.int64)
    out = []
    for name in ("k", "v"):
        x = e4m3_decode(cache[name][pids]) * cache[name + "_scale"][pids].astype(np.float64)[:, :, None, None]
        x = x.transpose(1, 0, 2, 3)
        out.append(x.reshape(x.shape[0], -1, x.shape[3])[:, :n_kv])
    return out


def attend(q, cache, table, q_start, kv_len, causal, scale, selected=None):
    """fp64 attention of q [T, Hq, d]: (O, L, A, D) with A = sum_j P_j |V_j| and
    D [T, Hq] = max_j scale * sum_c |q_c k_jc| over the visible keys (for error
    bounds).  Rows behind the last sequence stay NaN."""
    T, hq, d = q.shape
    hkv, page = cache["k"].shape[1], cache["k"].shape[2]
    g = hq // hkv
    O, A = np.full((T, hq, d), np.nan), np.full((T, hq, d), np.nan)
    L, D = np.full((T, hq), np.nan), np.full((T, hq), np.nan)
    for b in range(len(kv_len)):
        r0, r1, n_kv = int(q_start[b]), int(q_start[b + 1]), int(kv_len[b])
        if r1 == r0:
            continue
        k, v = cached_values(cache, table[b], n_kv)
        for row in range(r0, r1):
            pos = n_kv - (r1 - r0) + row - r0
            lim = max(0, min(n_kv, pos + 1)) if causal else n_kv
            for h in range(hkv):
                if selected is None:
                    keys = np.arange(lim)
                else:
                    keys = np.concatenate([np.arange(p * page, (p + 1) * page)
                                           for p in selected[row, h] if p >= 0] or [np.zeros(0, int)])
                    keys = keys[keys < lim].astype(int)
                rows = slice(h * g, (h + 1) * g)
                if len(keys) == 0:
                    O[row, rows], A[row, rows], L[row, rows], D[row, rows] = 0, 0, -np.inf, 0
                    continue
                kk, vv = k[h][keys], v[h][keys]
                s = q[row, rows].astype(np.float64) @ kk.T * scale
                m = s.max(axis=1, keepdims=True)
                p = np.exp(s - m)
                l = p.sum(axis=1, keepdims=True)
                p /= l
                O[row, rows], A[row, rows] = p @ vv, p @ np.abs(vv)
                L[row, rows] = (m + np.log(l))[:, 0]
                D[row, rows] = (np.abs(q[row, rows].astype(np.float64)) @ np.abs(kk).T).max(axis=1) * scale
    return O, L, A, D


def select(q, cache, table, q_start, kv_len, n_selected, n_first, n_recent):
    """int [T, Hkv, n_selected]; rows behind the last sequence hold -2."""
    T, hq, d = q.shape
    hkv, page = cache["k"].shape[1], cache["k"].shape[2]
    g = hq // hkv
    out = np.full((T, hkv, n_selected), -2, dtype=np.int32)
    for b in range(len(kv_len)):
        r0, r1, n_kv = int(q_start[b]), int(q_start[b + 1]), int(kv_len[b])
        for row in range(r0, r1):
            pos = n_kv - (r1 - r0) + row - r0
            n = pos // page + 1 if pos >= 0 else 0
            for h in range(hkv):
                x = q[row, h * g:(h + 1) * g].astype(F)
                amax = np.abs(x).max()
                inv = F(127.0) / F(amax) if amax >= 2.0 ** -100 else F(0)
                q8 = np.rint((x * F(inv)).astype(F)).astype(np.int64)
                up, down = np.maximum(q8, 0).sum(axis=0), np.minimum(q8, 0).sum(axis=0)
                pids = np.asarray(table[b, :n], dtype=np.int64)
                bd = cache["bounds"][pids, h].astype(np.int64)
                whole = bd[:, 1] @ up + bd[:, 0] @ down
                score = (whole.astype(F) * cache["k_scale"][pids, h]).astype(F)
                score[:n_first] = np.inf
                score[max(0, n - n_recent):] = np.inf
                top = np.sort(np.argsort(-score.astype(np.float64), kind="stable")[:n_selected])
                out[row, h] = -1
                out[row, h, :len(top)] = top
    return out
