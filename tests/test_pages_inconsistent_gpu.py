"""Compaction of a pool whose counts, tables and lengths do not agree: what is wrong is
reported and left as it is, whatever the workspace held, and the rest is moved."""

import numpy as np
import pytest
import torch

import exact_attention_fattn_gb300 as F
import oracle
from exact_attention_fattn_gb300 import _lib

pytestmark = pytest.mark.gpu
PAGES, ROWS, WIDTH, PAGE = 60, 5, 6, 32


class Pool:
    def __init__(self, seed):
        r = np.random.default_rng(seed)
        data = torch.from_numpy(r.integers(-9, 9, (PAGES, PAGE, 320)).astype(np.float32)).to(torch.bfloat16).cuda()
        self.cache = F.LatentCache(data, 256)
        self.kv = r.integers(1, WIDTH * PAGE, ROWS)
        self.table, self.refs = np.full((ROWS, WIDTH), -1), np.zeros(PAGES, int)
        free = list(r.permutation(PAGES))
        for b, n in enumerate(self.kv):
            for i in range(-(-n // PAGE)):
                self.table[b, i] = free.pop()
                self.refs[self.table[b, i]] = 1

    def entries(self):
        return [(b, i) for b, n in enumerate(self.kv) for i in range(-(-n // PAGE))]

    def compact(self, fill):
        """Both sides; the workspace full of one number.  Returns the status."""
        dev = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
        need = F.fattn_pages_workspace_bytes(PAGES, ROWS)
        ws = torch.full((need // 4,), fill, dtype=torch.int32, device="cuda").view(torch.uint8)
        t, kv, pool = dev(self.table), dev(self.kv), F.PagePool(dev(self.refs))
        planes = [self.cache.data.view(torch.int16).cpu().numpy().copy()]
        F.fattn_pages_compact(pool, self.cache, t, kv, workspace=ws)
        rc = F.fattn_check_status()
        oracle.pages.compact(self.refs, self.table, planes, PAGE, self.kv)
        assert np.array_equal(t.cpu().numpy(), self.table) and np.array_equal(pool.refs.cpu().numpy(), self.refs)
        assert np.array_equal(self.cache.data.view(torch.int16).cpu().numpy(), planes[0])
        assert np.array_equal(kv.cpu().numpy(), self.kv)
        return rc


@pytest.mark.parametrize("fill", [0, 1, 3, -1, 1 << 30])
def test_entries_whose_page_has_no_count(fill):
    """A page that was freed once too often, above and below the limit."""
    for seed in range(6):
        for above in (True, False):
            p = Pool(seed)
            limit = int((p.refs > 0).sum())
            some = [(b, i) for b, i in p.entries() if (p.table[b, i] >= limit) == above]
            b, i = some[seed % len(some)]
            page = int(p.table[b, i])
            p.refs[page] = 0
            if page == limit - 1:
                continue                        # the limit has moved below it
            assert p.compact(fill) == _lib.FATTN_ERR_BAD_INDEX, (seed, above)
            assert p.table[b, i] == page


@pytest.mark.parametrize("fill", [0, -1])
def test_consistent_pools(fill):
    for seed in range(20, 26):
        assert Pool(seed).compact(fill) == 0


@pytest.mark.parametrize("length", [-1, WIDTH * PAGE + 1, -(1 << 31)])
def test_lengths_that_make_no_sense_move_nothing(length):
    """The pages of such a sequence would move without its entries, so none does."""
    for row in (0, ROWS - 1):
        p = Pool(7)
        p.kv[row] = length
        assert p.compact(0) == _lib.FATTN_ERR_BAD_INDEX


def test_a_length_that_is_too_long():
    """Entries beyond what the sequence holds: pages that others hold are followed, free ones
    and those outside the pool are reported."""
    p = Pool(9)
    b = int(np.argmin(p.kv))
    n = -(-int(p.kv[b]) // PAGE)
    assert n < WIDTH
    p.table[b, n:] = PAGES + 5
    p.kv[b] = n * PAGE + 1
    assert p.compact(0) == _lib.FATTN_ERR_BAD_INDEX
    p = Pool(9)
    p.table[b, n] = max(x for x in range(PAGES) if p.refs[x] == 0)
    p.kv[b] = n * PAGE + 1
    assert p.compact(2) == _lib.FATTN_ERR_BAD_INDEX
