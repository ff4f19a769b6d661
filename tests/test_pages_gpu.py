"""The pages of a cache on the GPU: counts, tables, lengths and every plane of both
caches against the oracle's one sequence after the other, and what the calls
refuse or report."""

import ctypes

import numpy as np
import pytest
import torch

import exact_attention_fattn_gb300 as F
import oracle
from exact_attention_fattn_gb300 import _lib

pytestmark = pytest.mark.gpu
P = oracle.pages


def ok():
    assert F.fattn_check_status() == 0


class Pool:
    """A cache of either kind with random contents, as arrays and on the GPU."""

    def __init__(self, kind, pages, rows, max_pages, page, seed=0, gap=0, heads=3, bounds=True):
        r = np.random.default_rng(seed)
        self.page, self.rows, self.max_pages, self.pages = page, rows, max_pages, pages
        if kind == "latent":
            x = torch.from_numpy(r.integers(-9, 9, (pages, page, 320)).astype(np.float32)).to(torch.bfloat16).cuda()
            if gap:
                slab = torch.zeros((pages, page * 320 + gap), dtype=torch.bfloat16, device="cuda")
                y = slab[:, :page * 320].unflatten(1, (page, 320))
                y.copy_(x)
                x = y
            self.cache = F.LatentCache(x, 256)
            self.tensors = [x]
        else:
            k, v = (torch.from_numpy(r.integers(0, 256, (pages, heads, page, 64)).astype(np.uint8)).cuda() for _ in range(2))
            ks, vs = (torch.from_numpy(r.standard_normal((pages, heads)).astype(np.float32)).cuda() for _ in range(2))
            kb = torch.from_numpy(r.integers(-127, 128, (pages, heads, 2, 64)).astype(np.int8)).cuda() if bounds else None
            self.cache = F.Fp8Cache(k, v, ks, vs, kb)
            self.tensors = [x for x in self.cache if x is not None]
        self.pool = F.fattn_pages_alloc(self.cache)
        self.table = torch.full((rows, max_pages), -1, dtype=torch.int32, device="cuda")
        self.kv = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.h_planes = [x.view(torch.int16).cpu().numpy().copy() if x.dtype is torch.bfloat16 else x.cpu().numpy().copy()
                         for x in self.tensors]
        self.h_refs, self.h_table = np.zeros(pages, int), np.full((rows, max_pages), -1)
        self.h_kv = np.zeros(rows, int)

    def dev(self, x):
        return torch.tensor([int(i) for i in x], dtype=torch.int32, device="cuda")

    def fork(self, parent, child):
        F.fattn_pages_fork(self.pool, self.cache, self.table, self.kv, self.dev(parent), self.dev(child))
        return P.fork(self.h_refs, self.h_table, self.h_kv, self.page, parent, child)

    def extend(self, new, **kw):
        new = np.asarray(new)
        F.fattn_pages_extend(self.pool, self.cache, self.table, self.kv, self.dev(new), **kw)
        fine = P.extend(self.h_refs, self.h_table, self.h_planes, self.page, self.h_kv, new)
        if fine:
            self.kv.copy_(self.dev(new))
            self.h_kv = new.copy()
        return fine

    def free(self, rows):
        F.fattn_pages_free(self.pool, self.cache, self.table, self.kv, self.dev(rows))
        P.free(self.h_refs, self.h_table, self.h_kv, self.page, rows)

    def compact(self, **kw):
        F.fattn_pages_compact(self.pool, self.cache, self.table, self.kv, **kw)
        P.compact(self.h_refs, self.h_table, self.h_planes, self.page, self.h_kv)

    def same(self):
        assert np.array_equal(self.pool.refs.cpu().numpy(), self.h_refs)
        assert np.array_equal(self.table.cpu().numpy(), self.h_table)
        assert np.array_equal(self.kv.cpu().numpy(), self.h_kv)
        for x, y in zip(self.tensors, self.h_planes):
            x = x.view(torch.int16) if x.dtype is torch.bfloat16 else x
            assert np.array_equal(x.cpu().numpy(), y, equal_nan=True)


KINDS = [dict(kind="latent"), dict(kind="latent", gap=64), dict(kind="fp8"), dict(kind="fp8", heads=1, bounds=False)]


@pytest.mark.parametrize("page", [32, 64, 128])
@pytest.mark.parametrize("kw", KINDS)
def test_a_life(kw, page):
    """Prompts, samples of them, growth token by token and by pieces, ends, compaction."""
    p = Pool(pages=150, rows=12, max_pages=20, page=page, seed=page, **kw)
    assert p.extend([3 * page + 5, 2 * page, 1, page - 1, 4 * page + 1, 0, 0, 0, 0, 0, 0, 0])
    p.same()
    assert p.fork([0, 0, 1, 2, 4], [5, 6, 7, 8, 9])
    p.same()
    assert p.extend(p.h_kv + np.array([1, 1, 1, 1, 0, 1, 1, 0, 1, 3 * page, 0, 0]))
    p.same()
    assert p.extend(p.h_kv + np.array([40, 0, 7, 0, 1, page, 2, 1, 100, 0, 0, 77]))
    p.same()
    p.free([5, 1, 9, 5])
    p.same()
    p.compact()
    p.same()
    assert p.fork([0], [9]) and p.fork([9], [1])
    p.same()
    assert p.extend(p.h_kv + 3)
    p.free(list(range(12)))
    p.same()
    p.compact()
    p.same()
    assert not p.h_refs.any()
    ok()


def test_all_who_share_write_at_once():
    """Of those that write to one page the last keeps it if nobody else names it."""
    for idle in (False, True):
        p = Pool("latent", 60, 8, 5, 32, seed=1)
        assert p.extend([40, 0, 0, 0, 0, 0, 0, 0])
        p.fork([0] * 5, [6, 1, 4, 2, 7])
        page = int(p.h_table[0, 1])
        grow = np.where(p.h_kv > 0, 1, 0)
        if idle:
            grow[4] = 0
        assert p.extend(p.h_kv + grow)
        p.same()
        assert p.h_refs[page] == 1 and (p.h_table[4 if idle else 7, 1] == page)
    ok()


def test_many_sequences_and_pages():
    """More sequences than threads, more pages than one turn's, long growth."""
    r = np.random.default_rng(2)
    p = Pool("fp8", 40000, 4096, 130, 32, seed=2, heads=1, bounds=False)
    p.extend(np.where(np.arange(4096) % 5 == 0, r.integers(1, 200, 4096), 0))
    p.same()
    par = np.arange(0, 4090, 5)
    assert p.fork(np.tile(par, 3), np.concatenate([par + 1, par + 2, par + 4]))
    p.same()
    grow = r.integers(0, 3, 4096)
    grow[17], grow[4000], grow[1001] = 4000, 333, 3000
    assert p.extend(p.h_kv + grow)
    p.same()
    p.free(r.permutation(4096)[:2500])
    p.same()
    p.compact()
    p.same()
    ok()


def test_a_pool_of_a_million_pages():
    pages = 1 << 20
    p = Pool("fp8", pages, 2, 8, 32, seed=3, heads=1, bounds=False)
    refs = torch.ones(pages, dtype=torch.int32, device="cuda")
    hole = [5, 16383, 16384, 700001, pages - 1]
    refs[torch.tensor(hole, device="cuda")] = 0
    p.pool.refs.copy_(refs)
    p.h_refs[:] = 1
    p.h_refs[hole] = 0
    assert p.extend([100, 20])
    p.same()
    assert p.h_table[0, :4].tolist() == hole[:4] and p.h_table[1, 0] == hole[4]
    ok()


def test_too_few_pages():
    """Nobody gets any, entries to be filled become -1, and it is reported; one page
    less of demand is granted."""
    p = Pool("latent", 8, 4, 6, 32, seed=4)
    assert p.extend([70, 64, 0, 0])               # 3 + 2 pages
    p.fork([0], [2])
    assert not p.extend([97, 65, 71, 1])          # a copy and one, one, none (it keeps the page), one: 4 of 3
    assert F.fattn_check_status() == _lib.FATTN_ERR_NO_PAGES
    p.same()
    assert (p.h_table[0, 3], p.h_table[1, 2], p.h_table[3, 0]) == (-1, -1, -1)
    assert p.extend([97, 65, 71, 0])
    p.same()
    assert not p.extend([6 * 32, 6 * 32, 6 * 32, 6 * 32])   # more than the pool has at all
    assert F.fattn_check_status() == _lib.FATTN_ERR_NO_PAGES
    p.same()
    p.compact()                                    # nothing to move
    p.same()
    ok()


def test_forks_that_are_refused():
    """Children that are not empty, named twice, out of range or parents themselves
    are left as they are and reported; the others are taken."""
    for parent, child in (([0, 0], [3, 3]), ([0, 3], [3, 4]), ([0, 0, 1], [-1, 8, 5]), ([9, 0], [3, 4]), ([0, 1], [1, 2]), ([0], [0])):
        p = Pool("fp8", 30, 8, 5, 32, seed=5)
        assert p.extend([70, 64, 0, 0, 0, 0, 0, 0])
        assert not p.fork(parent, child)
        assert F.fattn_check_status() == _lib.FATTN_ERR_BAD_INDEX, (parent, child)
        p.same()
    ok()


def test_senseless_numbers():
    p = Pool("latent", 30, 4, 5, 32, seed=6)
    assert p.extend([70, 64, 33, 0])
    # lengths that shrink, are negative or past the table: that sequence gets nothing, the others do
    for b, new in ((0, 69), (1, -5), (2, 5 * 32 + 1)):
        n = p.h_kv.copy()
        n[3] += 40
        n[b] = new
        F.fattn_pages_extend(p.pool, p.cache, p.table, p.kv, p.dev(n))
        assert F.fattn_check_status() == _lib.FATTN_ERR_BAD_INDEX
        n[b] = p.h_kv[b]
        P.extend(p.h_refs, p.h_table, p.h_planes, p.page, p.h_kv, n)
        p.h_kv = n
        p.kv.copy_(p.dev(n))
        p.same()
    # rows out of range; pages freed that were free
    F.fattn_pages_free(p.pool, p.cache, p.table, p.kv, p.dev([7, -1, 1]))
    assert F.fattn_check_status() == _lib.FATTN_ERR_BAD_INDEX
    P.free(p.h_refs, p.h_table, p.h_kv, p.page, [1])
    p.same()
    page = int(p.h_table[0, 0])
    p.pool.refs[page] = 0
    F.fattn_pages_free(p.pool, p.cache, p.table, p.kv, p.dev([0]))
    assert F.fattn_check_status() == _lib.FATTN_ERR_BAD_INDEX
    assert int(p.pool.refs[page]) == 0 and int(p.pool.refs.min()) == 0
    # an entry outside the pool: of a sequence that grows, forks or is compacted
    p = Pool("latent", 30, 4, 5, 32, seed=6)
    assert p.extend([70, 64, 33, 0])
    p.table[0, 2] = 1 << 20
    before = [x.clone() for x in p.tensors]
    for call in (lambda: F.fattn_pages_extend(p.pool, p.cache, p.table, p.kv, p.kv + 1),
                 lambda: F.fattn_pages_fork(p.pool, p.cache, p.table, p.kv, p.dev([0]), p.dev([3])),
                 lambda: F.fattn_pages_free(p.pool, p.cache, p.table, p.kv, p.dev([3]))):
        call()
        assert F.fattn_check_status() == _lib.FATTN_ERR_BAD_INDEX
    assert all(torch.equal(x, y) for x, y in zip(p.tensors, before))
    p.pool.refs[0] = 0
    F.fattn_pages_compact(p.pool, p.cache, p.table, p.kv)
    assert F.fattn_check_status() == _lib.FATTN_ERR_BAD_INDEX
    ok()


def test_captured_steps_replay_on_other_lengths():
    """Fork, room and freeing in one graph, replayed from other states; the workspace is
    shared by two graphs that are replayed in turn."""
    ws = torch.full((F.fattn_pages_workspace_bytes(60, 6),), 0x7F, dtype=torch.uint8, device="cuda")
    p = Pool("fp8", 60, 6, 8, 32, seed=7)
    parent, child, step = p.dev([0, 1]), p.dev([3, 4]), p.dev([1] * 6)
    new = torch.zeros(6, dtype=torch.int32, device="cuda")

    def grow():
        torch.add(p.kv, step, out=new)
        F.fattn_pages_extend(p.pool, p.cache, p.table, p.kv, new, workspace=ws)
        p.kv.copy_(new)

    p.extend([33, 5, 0, 0, 0, 0])
    p.same()
    graphs = []
    for what in (lambda: F.fattn_pages_fork(p.pool, p.cache, p.table, p.kv, parent, child), grow,
                 lambda: F.fattn_pages_free(p.pool, p.cache, p.table, p.kv, child),
                 lambda: F.fattn_pages_compact(p.pool, p.cache, p.table, p.kv, workspace=ws)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            what()
        graphs.append(g)
    for n in (1, 0, 40, 31, 3):
        graphs[0].replay()
        P.fork(p.h_refs, p.h_table, p.h_kv, 32, [0, 1], [3, 4])
        step.fill_(n)
        graphs[1].replay()
        assert P.extend(p.h_refs, p.h_table, p.h_planes, 32, p.h_kv, p.h_kv + n)
        p.h_kv = p.h_kv + n
        p.same()
        graphs[2].replay()
        P.free(p.h_refs, p.h_table, p.h_kv, 32, [3, 4])
        graphs[3].replay()
        P.compact(p.h_refs, p.h_table, p.h_planes, 32, p.h_kv)
        p.same()
    ok()


def test_large_pages_past_32_bits():
    """Copies between pages whose offsets pass 2^32 bytes."""
    data = torch.zeros((62000, 64, 576), dtype=torch.bfloat16, device="cuda")
    cache = F.LatentCache(data, 512)
    pool = F.fattn_pages_alloc(cache)
    pool.refs.fill_(1)
    pool.refs[61999] = pool.refs[7] = 0
    table = torch.full((2, 2), 61000, dtype=torch.int32, device="cuda")
    kv = torch.tensor([10, 0], dtype=torch.int32, device="cuda")
    data[61000] = torch.randn(64, 576, device="cuda").to(torch.bfloat16)
    F.fattn_pages_fork(pool, cache, table, kv, kv[1:], torch.ones(1, dtype=torch.int32, device="cuda"))
    F.fattn_pages_extend(pool, cache, table, kv, kv + 1)
    ok()
    assert table.tolist() == [[7, 61000], [61000, 61000]] and torch.equal(data[7], data[61000])
    F.fattn_pages_free(pool, cache, table, kv, torch.zeros(1, dtype=torch.int32, device="cuda"))
    F.fattn_pages_compact(pool, cache, table, kv)      # two holes, 7 and 61999; 61998 moves to 7
    ok()
    assert int(pool.refs[61999]) == 0 and int(pool.refs[61998]) == 0 and int((pool.refs == 0).sum()) == 2
    assert int(pool.refs[7]) == 1


@pytest.mark.parametrize("seed", [0, 1, 2])
def test_planes_of_any_size(seed):
    """Through the C ABI: parts of a page of a few bytes up to several pieces, aligned to
    4, 8 or 16 bytes, with gaps between the pages that stay as they were."""
    r = np.random.default_rng(90 + seed)
    pages, B, width = 300, 9, 20
    sizes = [[4, 2048, 16400, 70000, 131072], [2032, 2064, 16384, 32, 49156], [100000, 16, 8, 65536, 4100]][seed]
    aligns = [[4, 16, 16, 16, 16], [16, 16, 16, 16, 4], [16, 16, 8, 4, 16]][seed]
    gaps = [int(x) for x in r.integers(0, 5, 5) * 16]
    bufs, planes, want = [], [], []
    for size, align, gap in zip(sizes, aligns, gaps):
        stride = size + gap + (-(size + gap)) % align
        buf = torch.from_numpy(r.integers(0, 256, 16 + pages * stride).astype(np.uint8)).cuda()
        base = align % 16                                # 16-byte aligned, or 4 or 8 bytes further
        bufs.append((buf, base, stride, size))
        planes.append((buf.data_ptr() + base, stride, size))
        want.append(buf.cpu().numpy().copy())
    held = r.permutation(pages)[:B * 10].reshape(B, 10)
    table = np.full((B, width), -1)
    table[:, :10] = held
    refs = np.zeros(pages, int)
    refs[held] = 1
    kv = np.full(B, 10 * 32 - 5)
    d_table, d_refs, d_kv = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (table, refs, kv))
    lib = _lib.load()
    need = int(lib.fattn_pages_workspace_bytes(pages, B))
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    pool = _lib.PagePoolStruct(d_refs.data_ptr(), pages, 32)
    arr = (_lib.PlaneStruct * 5)(*planes)
    assert lib.fattn_pages_compact(ctypes.byref(pool), arr, 5, d_table.data_ptr(), d_kv.data_ptr(), ws.data_ptr(), need, B,
                                   width, torch.cuda.current_stream().cuda_stream) == 0
    ok()
    views = [np.lib.stride_tricks.as_strided(w[base:], (pages, size), (stride, 1)) for w, (_, base, stride, size) in zip(want, bufs)]
    P.compact(refs, table, views, 32, kv)
    assert np.array_equal(d_table.cpu().numpy(), table) and np.array_equal(d_refs.cpu().numpy(), refs)
    for w, (buf, *_) in zip(want, bufs):
        assert np.array_equal(buf.cpu().numpy(), w)


def test_a_wait_budget_that_runs_out():
    """Copies that give up are reported, and the next call is right."""
    for i in range(3):
        p = Pool("latent", 400, 20, 12, 128, seed=i)
        p.extend([100 + 50 * j for j in range(20)])
        p.free(list(range(0, 20, 2)))
        F.fattn_set_wait_budget(1)
        try:
            F.fattn_pages_compact(p.pool, p.cache, p.table, p.kv)
            assert F.fattn_check_status() in (_lib.FATTN_OK, _lib.FATTN_ERR_TIMEOUT)
        finally:
            F.fattn_set_wait_budget(0)
    p = Pool("latent", 400, 20, 12, 128, seed=5)
    p.extend([100 + 50 * j for j in range(20)])
    p.free(list(range(0, 20, 2)))
    p.compact()
    p.same()
    ok()


def test_refusals_of_the_binding():
    p = Pool("latent", 10, 3, 4, 32)
    i = p.dev([0])
    good = dict(pool=p.pool, cache=p.cache, table=p.table, kv=p.kv)
    for bad in (dict(pool=F.PagePool(p.pool.refs[:5])), dict(pool=F.PagePool(p.pool.refs.float())), dict(cache=p.cache.data),
                dict(table=p.table.long()), dict(table=p.table[0]), dict(table=p.table.t()), dict(kv=p.kv[:2]), dict(kv=p.kv.cpu())):
        a = {**good, **bad}
        for call in (lambda: F.fattn_pages_fork(a["pool"], a["cache"], a["table"], a["kv"], i, i),
                     lambda: F.fattn_pages_extend(a["pool"], a["cache"], a["table"], a["kv"], p.kv),
                     lambda: F.fattn_pages_free(a["pool"], a["cache"], a["table"], a["kv"], i),
                     lambda: F.fattn_pages_compact(a["pool"], a["cache"], a["table"], a["kv"])):
            with pytest.raises((TypeError, ValueError)):
                call()
    with pytest.raises(ValueError):
        F.fattn_pages_fork(p.pool, p.cache, p.table, p.kv, p.dev([0, 1]), i)
    with pytest.raises(_lib.FattnError):
        F.fattn_pages_fork(p.pool, p.cache, p.table, p.kv, p.dev([0, 1, 0, 1]), p.dev([2, 2, 2, 2]))
    with pytest.raises(_lib.FattnError):
        F.fattn_pages_compact(p.pool, p.cache, p.table, p.kv, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    empty = p.dev([])
    F.fattn_pages_fork(p.pool, p.cache, p.table, p.kv, empty, empty)
    F.fattn_pages_free(p.pool, p.cache, p.table, p.kv, empty)
    ok()
