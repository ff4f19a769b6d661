"""A pool without enough pages, in the middle of captured steps that make room, append and
attend: what sequences share stays as it was, those that have room go on, and the
host learns which were left out."""

import numpy as np
import pytest
import torch

import exact_attention_fattn_gb300 as F
import oracle
from exact_attention_fattn_gb300 import _lib

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.tensor([int(i) for i in x], dtype=torch.int32, device="cuda")


def planes(kind, cache):
    return [cache.data.view(torch.int16)] if kind == "latent" else [x for x in cache if x is not None]


class Server:
    """Four sequences on a cache of either kind; 1 is a copy of 0 that shares its pages."""

    def __init__(self, kind, pages, lens, page=32):
        torch.manual_seed(3)
        self.kind, self.page = kind, page
        self.cache = F.fattn_latent_alloc(pages, 256, page) if kind == "latent" else F.fattn_cache_alloc(pages, 2, 64, page)
        self.pool = F.fattn_pages_alloc(self.cache)
        self.table = torch.full((4, 6), -1, dtype=torch.int32, device="cuda")
        self.kv = torch.zeros(4, dtype=torch.int32, device="cuda")
        self.new, self.qs = torch.zeros_like(self.kv), torch.zeros(5, dtype=torch.int32, device="cuda")
        self.make(8 * 6 * page)
        self.o = self.l = None
        self.step([lens[0], 0, lens[2], lens[3]])
        F.fattn_pages_fork(self.pool, self.cache, self.table, self.kv, dev([0]), dev([1]))
        assert F.fattn_check_status() == 0

    def make(self, rows):
        rnd = lambda *s: torch.randn(*s, device="cuda").to(torch.bfloat16)
        self.lat, self.key, self.q = rnd(rows, 256), rnd(rows, 64), rnd(rows, 3, 320)
        self.k, self.v, self.q8 = rnd(rows, 2, 64), rnd(rows, 2, 64), rnd(rows, 4, 64)

    def ask(self, grow):
        self.qs.copy_(dev([0, *np.cumsum(grow)]))
        self.new.copy_(self.kv + dev(grow))

    def call(self, T):
        F.fattn_pages_extend(self.pool, self.cache, self.table, self.kv, self.new)
        if self.kind == "latent":
            F.fattn_latent_append(self.lat[:T], self.key[:T], self.cache, self.table, self.qs, self.new)
            return F.fattn_latent_fwd(self.q[:T], self.cache, self.table, self.qs, self.new, scale=0.1, out=self.o, lse=self.l)
        F.fattn_cache_append(self.k[:T], self.v[:T], self.cache, self.table, self.qs, self.new)
        return F.fattn_cache_fwd(self.q8[:T], self.cache, self.table, self.qs, self.new, out=self.o, lse=self.l)

    def step(self, grow):
        self.ask(grow)
        self.call(sum(grow))
        self.kv.copy_(self.new)


@pytest.mark.parametrize("kind", ["latent", "fp8"])
def test_a_captured_step_on_a_pool_that_is_too_small(kind):
    """0 and 1 would write into the page that they share, 2 needs a new one, 3 has room in its own;
    no page is free.  Nothing that 0, 1 and 2 have changes, and 3 gets its token."""
    s = Server(kind, 5, [40, 0, 64, 20])                # 2 + 2 + 1 pages
    assert int((s.pool.refs == 0).sum()) == 0
    T = 4
    T_o = (T, 3, 256) if kind == "latent" else (T, 4, 64)
    s.o, s.l = torch.full(T_o, 7.0, dtype=torch.bfloat16, device="cuda"), torch.full(T_o[:2], 7.0, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.call(T)
    s.ask([1, 1, 1, 1])
    before = [x.clone() for x in planes(kind, s.cache)]
    tables, refs = s.table.clone(), s.pool.refs.clone()
    g.replay()
    assert F.fattn_check_status() == _lib.FATTN_ERR_NO_PAGES
    assert s.new.tolist() == [-1, -1, -1, 21] and s.kv.tolist() == [40, 40, 64, 20]
    assert torch.equal(s.pool.refs, refs) and torch.equal(s.table[:2], tables[:2])
    own = int(tables[3, 0])
    rest = [p for p in range(5) if p != own]
    for x, y in zip(planes(kind, s.cache), before):
        assert torch.equal(x[rest], y[rest])
    assert any(not torch.equal(x[own], y[own]) for x, y in zip(planes(kind, s.cache), before))
    assert bool((s.o[:3] == 7.0).all()) and bool((s.l[:3] == 7.0).all())
    assert bool(torch.isfinite(s.l[3]).all()) and bool((s.l[3] != 7.0).any())

    # The host takes up what went on, ends sequence 2, and asks again for the others.
    s.kv.copy_(torch.maximum(s.kv, s.new))
    F.fattn_pages_free(s.pool, s.cache, s.table, s.kv, dev([2]))
    s.ask([1, 1, 2, 0])
    g.replay()
    assert F.fattn_check_status() == 0
    assert s.new.tolist() == [41, 41, 2, 21]
    assert s.table[0, 0] == s.table[1, 0] and s.table[0, 1] != s.table[1, 1]
    # each has its own token behind the same forty
    a, b = (planes(kind, s.cache)[0][int(s.table[i, 1])] for i in (0, 1))
    at = (slice(0, 8),) if kind == "latent" else (slice(None), slice(0, 8))
    tok = (8,) if kind == "latent" else (slice(None), 8)
    if kind == "latent":
        assert torch.equal(a[at], b[at])
        assert torch.equal(a[tok][:256], s.lat[0].view(torch.int16)) and torch.equal(b[tok][:256], s.lat[1].view(torch.int16))
    assert not torch.equal(a[tok], b[tok])


def test_which_sequences_are_left_out():
    """Random pools: refused, the sequences that lack room have length -1 and the others keep
    theirs; granted, all lengths stay.  The tables and counts are the oracle's."""
    r = np.random.default_rng(8)
    refused = 0
    for n in range(30):
        rows, page, pages = 9, 32, 26
        cache = F.fattn_latent_alloc(pages, 256, page)
        pool = F.fattn_pages_alloc(cache)
        refs, table, kv = np.zeros(pages, int), np.full((rows, 7), -1), np.zeros(rows, int)
        first = np.where(np.arange(rows) < 5, r.integers(1, 110, rows), 0)
        assert oracle.pages.extend(refs, table, [], page, kv, first.copy())
        kv[:] = first
        assert oracle.pages.fork(refs, table, kv, page, [0, 0, 1], [5, 6, 7])
        grow = r.integers(0, [2, 40, 100][n % 3], rows)
        new = kv + grow
        new[8] = 40 if n % 4 else 0
        d_table, d_kv, d_new = torch.tensor(table, dtype=torch.int32, device="cuda"), dev(kv), dev(new)
        pool.refs.copy_(dev(refs))
        F.fattn_pages_extend(pool, cache, d_table, d_kv, d_new)
        asked = new.copy()
        fine = oracle.pages.extend(refs, table, [], page, kv, new)
        assert F.fattn_check_status() == (0 if fine else _lib.FATTN_ERR_NO_PAGES)
        refused += not fine
        assert fine or (new != asked).any()
        assert d_new.tolist() == new.tolist() and d_kv.tolist() == kv.tolist()
        assert np.array_equal(d_table.cpu().numpy(), table) and np.array_equal(pool.refs.cpu().numpy(), refs)
    assert 5 <= refused <= 25


def test_senseless_lengths_are_left_out_too():
    cache = F.fattn_latent_alloc(12, 256, 32)
    pool = F.fattn_pages_alloc(cache)
    table = torch.full((4, 3), -1, dtype=torch.int32, device="cuda")
    for old, new, want in (([0, 5, -1, 0], [3, 4, 7, 9], [3, -1, -1, 9]), ([3, 0, 0, 9], [4, 97, -5, 96], [4, -1, -1, 96])):
        d = dev(new)
        F.fattn_pages_extend(pool, cache, table, dev(old), d)
        assert F.fattn_check_status() == _lib.FATTN_ERR_BAD_INDEX
        assert d.tolist() == want
