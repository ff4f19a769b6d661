"""Seeded ragged batches over a paged latent cache, and the error bounds of the
attention over it, shared by the latent cache's tests."""

import copy

import numpy as np
import torch

import oracle
from cache_util import to_bf16
from exact_attention_fattn_gb300.latent import LatentCache

BF16_STEP = 2.0 ** -8      # half a step, relative to the value
ROPE = 64


class LatentBatch:
    """lens: tokens cached per sequence; news: new ones among them.  Pages are a
    random permutation; slots behind a sequence's end and unused pages hold NaN,
    and unused table entries a page far outside."""

    def __init__(self, seed, lens, news, heads, rank, page, pad_rows=0, spare=2, scale_q=1.0, whole=False):
        r = np.random.default_rng(seed)
        self.lens, self.news, self.heads, self.rank, self.page = lens, news, heads, rank, page
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
        width = rank + ROPE
        if whole:       # small whole numbers
            self.data = r.integers(-8, 9, (self.pages, page, width)).astype(np.float32)
        else:
            gain = np.exp(0.4 * r.standard_normal(width))
            self.data = to_bf16(r.standard_normal((self.pages, page, width)) * gain)
        for b, t in enumerate(lens):
            for i in range(t, n_pages[b] * page):
                self.data[self.table[b, i // page], i % page] = np.nan
        for p in perm[at:]:
            self.data[p] = np.nan
        self.q = to_bf16(scale_q * r.standard_normal((self.T, heads, width)))
        self.latent = to_bf16(r.standard_normal((self.T, rank)))
        self.k_rope = to_bf16(r.standard_normal((self.T, ROPE)))
        self.q_rope = to_bf16(r.standard_normal((self.T, heads, ROPE)))

    def tables(self):
        """This batch and, with more than 64 rows a sequence, itself with tables that
        have room for many more pages: that decides which kernel works on them."""
        yield self
        if self.rank == 512 and self.T * self.heads > 64 * len(self.lens):
            b = copy.copy(self)
            b.max_pages = self.table.shape[1] + 120000 // self.page
            b.table = np.full((len(self.lens), b.max_pages), 1 << 30, dtype=np.int32)
            b.table[:, :self.table.shape[1]] = self.table
            yield b

    def device(self, gap=0):
        """(cache, page_table, q_start, kv_len) on the GPU; gap: elements left
        between pages."""
        x = torch.from_numpy(self.data).to(torch.bfloat16).cuda()
        if gap:
            slab = torch.full((self.pages, x[0].numel() + gap), float("nan"), dtype=torch.bfloat16, device="cuda")
            y = slab[:, :x[0].numel()].unflatten(1, x.shape[1:])
            y.copy_(x)
            x = y
        return (LatentCache(x, self.rank), *(torch.from_numpy(a).cuda() for a in (self.table, self.q_start, self.kv_len)))

    def rows(self, x):
        return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).cuda()


def check_latent(o, lse, want, width):
    """o, lse: arrays; want: oracle.latent.attend's (O, L, A, D).

    A score is a sum of `width` products of bf16 numbers, exact in fp32, in any
    order with truncation: off by at most (width + 8) 2^-23 D; the scaling, the
    reference and the exponential add 2^-20.  With delta their sum, |dL| <= delta +
    2^-22 |L| (the logarithm).  A probability is rounded to bf16 once (2^-8) for the
    second product, whose sum's order costs less than delta, and the output once:
      |dO| <= 2^-8 |O| + (2^-8 + 2 delta) (A + |O|)."""
    O, L, A, D = want
    live = ~np.isnan(L)
    delta = (width + 8) * 2.0 ** -23 * D + 2.0 ** -20
    allow = BF16_STEP * np.abs(O) + (BF16_STEP + 2 * delta[..., None]) * (A + np.abs(O)) + 1e-38
    none = live & np.isneginf(L)
    assert np.isneginf(lse[none]).all() and (o[none] == 0).all()
    some = live & ~none
    err = np.abs(o - O)
    assert np.isfinite(o[some]).all()
    assert (err[some] <= allow[some]).all(), float((err[some] / allow[some]).max())
    dl = np.abs(lse[some] - L[some])
    assert (dl <= delta[some] + 2.0 ** -22 * np.abs(L[some])).all(), float(dl.max())
