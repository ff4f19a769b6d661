"""Seeded ragged batches over a paged cache, and the error bounds of the
attention over it, shared by the cache's tests."""

import numpy as np
import torch

import oracle
from exact_attention_fattn_gb300.cache import Fp8Cache

BF16_STEP, F16_STEP = 2.0 ** -8, 2.0 ** -11      # half a step, relative to the value


def to_bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).float().numpy()


class Batch:
    """lens: tokens cached per sequence; news: new ones among them.  The
    cache's pages are a random permutation; slots behind a sequence's end and
    unused pages hold NaN codes and unused table entries a page far outside."""

    def __init__(self, seed, lens, news, hkv, g, d, page, pad_rows=0, spread=2, spare=2, filled=True):
        r = np.random.default_rng(seed)
        self.lens, self.news, self.hkv, self.g, self.d, self.page = lens, news, hkv, g, d, page
        self.hq = hkv * g
        n_pages = [-(-t // page) for t in lens]
        self.pages = sum(n_pages) + spare
        self.max_pages = max(1, max(n_pages)) + 1
        perm = r.permutation(self.pages)
        self.table = np.full((len(lens), self.max_pages), 1 << 30, dtype=np.int32)
        at = 0
        for b, n in enumerate(n_pages):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.q_start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.kv_len = np.asarray(lens, dtype=np.int32)
        self.T = int(self.q_start[-1]) + pad_rows
        shape = (self.pages, hkv, page, d)
        self.cache = {"bounds": np.zeros((self.pages, hkv, 2, d), np.int8)}
        for name in ("k", "v"):
            e = r.integers(-spread, spread + 1, size=shape[:2])
            x = r.standard_normal(shape) * 100.0
            self.cache[name] = oracle.e4m3_encode(x.astype(np.float32))
            self.cache[name + "_scale"] = (2.0 ** (e - 6)).astype(np.float32)
        lo = np.floor(oracle.e4m3_decode(self.cache["k"]).astype(np.float32) * np.float32(127) / np.float32(448))
        hi = np.ceil(oracle.e4m3_decode(self.cache["k"]).astype(np.float32) * np.float32(127) / np.float32(448))
        self.cache["bounds"] = np.stack([lo.min(axis=2), hi.max(axis=2)], axis=2).astype(np.int8)
        used = np.zeros((self.pages, page), bool)
        for b, t in enumerate(lens):
            old = t if filled else max(0, t - news[b])
            for i in range(old):
                used[self.table[b, i // page], i % page] = True
        for name in ("k", "v"):
            self.cache[name][~np.broadcast_to(used[:, None, :, None], shape)] = 0x7F
        self.q = to_bf16(r.standard_normal((self.T, self.hq, d)))
        self.k_new = to_bf16(r.standard_normal((self.T, hkv, d)) * 2.0)
        self.v_new = to_bf16(r.standard_normal((self.T, hkv, d)))

    def device(self, page_gap=0):
        """(cache, page_table, q_start, kv_len) on the GPU; page_gap: bytes left
        between pages."""
        t = {}
        for name in ("k", "v"):
            x = torch.from_numpy(self.cache[name]).cuda()
            if page_gap:
                slab = torch.full((self.pages, x[0].numel() + page_gap), 0x7F, dtype=torch.uint8, device="cuda")
                y = slab[:, :x[0].numel()].unflatten(1, x.shape[1:])
                y.copy_(x)
                x = y
            t[name] = x
            t[name + "_scale"] = torch.from_numpy(self.cache[name + "_scale"]).cuda()
        c = Fp8Cache(t["k"], t["v"], t["k_scale"], t["v_scale"], torch.from_numpy(self.cache["bounds"]).cuda())
        return (c, *(torch.from_numpy(x).cuda() for x in (self.table, self.q_start, self.kv_len)))

    def rows(self, x):
        return torch.from_numpy(x).to(torch.bfloat16).cuda()


def check_attention(o, lse, want, d, amax_q, kmax):
    """o, lse: arrays; want: oracle.cache.attend's (O, L, A, D).

    A score s = scale sum_c q_c k_c is summed in fp32 from exact products of a
    code and a query's entry.  The entry is either its row's scaled by a power
    of two into fp16 (off by 2^-25 of the largest at most) or the sum of two
    e4m3 parts of the row scaled so that its largest is at least 224, off by at
    most half a subnormal step, 2^-10: 2^-17 of the largest.  A score is off by
    at most
      delta = (d + 8) 2^-23 D + 2^-17 scale amax_q sum_c |k_c| + 2^-20,
    the first term counting truncated sums, the last the exponential's own
    error.  A probability is rounded to fp16 once (2^-11) and the output to
    bf16 (2^-8): |dO| <= 2^-8 |O| + (2^-11 + 2 delta)(A + |O|) and |dL| <= delta
    + 2^-22 |L| (the logarithm).  fp16 probabilities below 2^-14 are off by at
    most 2^-25 of the largest: 2^-25 n |V|, below what A's term leaves."""
    O, L, A, D = want
    live = ~np.isnan(L)
    delta = (d + 8) * 2.0 ** -23 * D + 2.0 ** -17 * amax_q * kmax * d / np.sqrt(d) + 2.0 ** -20
    allow = BF16_STEP * np.abs(O) + (F16_STEP + 2 * delta[..., None]) * (A + np.abs(O)) + 2.0 ** -24 * np.nan_to_num(A).max()
    err = np.abs(o - O)
    assert np.isfinite(o[live]).all()
    assert (err[live] <= allow[live]).all(), float((err[live] / np.maximum(allow[live], 1e-300)).max())
    none = live & np.isneginf(L)
    assert np.isneginf(lse[none]).all() and (o[none] == 0).all()
    some = live & ~none
    dl = np.abs(lse[some] - L[some])
    assert (dl <= delta[some] + 2.0 ** -22 * np.abs(L[some])).all(), float(dl.max())
