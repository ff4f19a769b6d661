"""The paged cache as a server holds it: page tables for far more tokens than
any sequence has, pools larger than what is in use, batches that mix pieces of
prompts with single tokens, and batches drawn over all of the sizes.  Table
width and pool size decide between the attention's kernels, its grid and the
selection's kernels, so results are held to the oracle on both sides."""

import numpy as np
import pytest
import torch

import test_cache_gpu as T
from cache_util import Batch
from exact_attention_fattn_gb300 import cache as K

pytestmark = pytest.mark.gpu
C = T.C


def widen(b, columns):
    """The same batch under a table of `columns` entries; the new ones lie far
    outside the cache and are not to be read."""
    t = np.full((len(b.lens), columns), 1 << 30, dtype=np.int32)
    t[:, :b.max_pages] = b.table
    b.table, b.max_pages = t, columns
    return b


def in_pool(b, pages):
    """The same batch in the last pages of a cache of `pages`; the others hold zeros."""
    small = b.device

    def device(page_gap=0):
        c, table, qs, kl = small()
        big = K.fattn_cache_alloc(pages, b.hkv, b.d, b.page, bounds=True)
        for x, y in zip(big, c):
            x[pages - b.pages:] = y
        return big, torch.where(table < b.pages, table + (pages - b.pages), table), qs, kl

    b.device = device
    return b


@pytest.mark.parametrize("columns", [2048, 40000])
@pytest.mark.parametrize("pages", [None, 9000])
@pytest.mark.parametrize("d,lens,news,g", [
    (128, [1000], [1], 4), (128, [700, 90], [1, 1], 16),          # single tokens
    (128, [600, 300], [5, 4], 8), (64, [900], [24], 1),           # 2 to 4 units of rows a sequence
    (128, [500, 260], [200, 130], 2)])                            # prompts
def test_wide_tables_and_large_pools(d, lens, news, g, pages, columns):
    b = widen(Batch(500 + columns, lens, news, 2, g, d, 64), columns)
    if pages:
        in_pool(b, pages)
    T.check(b)
    for k in (4, 12):
        want = C.select(b.q, b.cache, b.table, b.q_start, b.kv_len, k, 1, 1)
        assert np.array_equal(T.run_select(b, k, 1, 1), want)
    T.check(b, selected=want)
    T.check_append(widen(Batch(501, lens, news, 2, g, d, 64, filled=False), columns), rope_dim=d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,news,g", [
    ([300] * 60 + [2000], [1] * 60 + [180], 4),       # the average is a single token's
    ([1500] + [260] * 6, [700] + [1] * 6, 4),         # the average is a prompt's
    ([500, 40, 900, 33, 1], [90, 0, 1, 33, 1], 8)])
def test_mixed_batches(d, lens, news, g):
    b = Batch(510 + d, lens, news, 2, g, d, 64, pad_rows=2)
    T.check(b)
    T.check(b, causal=False)
    sel = C.select(b.q, b.cache, b.table, b.q_start, b.kv_len, 6, 1, 2)
    assert np.array_equal(T.run_select(b, 6, 1, 2), sel)
    T.check(b, selected=sel)
    T.check_append(Batch(511 + d, lens, news, 2, g, d, 64, pad_rows=2, filled=False), rope_dim=d)


def draw(seed):
    """Sizes of one batch: sequences, lengths, rows, heads, page, spread of the
    scales, padding rows and bytes between pages."""
    r = np.random.default_rng(seed)
    pick = lambda *x: x[int(r.integers(len(x)))]
    B = pick(1, 1, 2, 3, 5, 9, 33, 70)
    cap = pick(40, 200, 1500, 6000) if B < 10 else pick(40, 300)
    g, most = pick(1, 2, 3, 4, 6, 8, 12, 16, 17, 24, 33, 64), pick(1, 1, 2, 5, 17, 60, 300)
    most = min(most, max(1, 6000 // (B * g)))
    lens = [int(x) for x in np.exp(r.uniform(0, np.log(cap), B))]
    news = [min(t, int(r.integers(0, most + 1))) for t in lens]
    if sum(news) == 0:
        news[0] = 1
    size = dict(lens=lens, news=news, hkv=pick(1, 2, 3, 5), g=g, d=pick(64, 128), page=pick(32, 64, 128),
                pad_rows=pick(0, 1, 3), spread=pick(0, 2, 12))
    return size, dict(causal=pick(True, True, False), page_gap=pick(0, 0, 16, 4096)), r


@pytest.mark.parametrize("seed", range(2000, 2040))
def test_attend_drawn(seed):
    size, kw, _ = draw(seed)
    T.check(Batch(seed, **size), **kw)


@pytest.mark.parametrize("seed", range(3000, 3030))
def test_select_and_attend_drawn(seed):
    size, kw, r = draw(seed)
    b = Batch(seed, **size)
    k = int(r.integers(1, 12))
    first = int(r.integers(0, k + 1))
    recent = int(r.integers(0, k - first + 1))
    want = C.select(b.q, b.cache, b.table, b.q_start, b.kv_len, k, first, recent)
    assert np.array_equal(T.run_select(b, k, first, recent), want)
    T.check(b, selected=np.maximum(want, -1), **kw)


@pytest.mark.parametrize("seed", range(4000, 4040))
def test_append_drawn(seed):
    size, kw, r = draw(seed)
    rope_dim = int(r.choice([0, 16, 32, 64, size["d"]]))
    T.check_append(Batch(seed, filled=False, **size), rope_dim, bool(r.random() < 0.5), with_q=bool(r.random() < 0.7),
                   bounds=bool(r.random() < 0.7), page_gap=kw["page_gap"])


def test_the_same_bits_from_calls_that_differ_in_nothing_else():
    """Output buffers, workspaces, row strides and page distances do not change a result."""
    for news in ([1, 1], [70, 30]):
        b = Batch(520, [900, 400], news, 2, 4, 128, 64)
        c, *where = b.device()
        q = b.rows(b.q)
        o, l = K.fattn_cache_fwd(q, c, *where)
        wide = torch.zeros((b.T, b.hq * b.d + 40), dtype=torch.bfloat16, device="cuda")
        wide[:, :b.hq * b.d] = q.flatten(1)
        c2, *_ = b.device(page_gap=32)
        ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
        o2, l2 = K.fattn_cache_fwd(wide[:, :b.hq * b.d].unflatten(1, (b.hq, b.d)), c2, *where, workspace=ws)
        assert torch.equal(o, o2) and torch.equal(l, l2)
    T.status_ok()
