"""The paged 8-bit cache on the GPU: appending and selecting bit for bit
against the oracle, attention within bounds derived from the arithmetic
(cache_util.check_attention), over head layouts, page sizes, ragged lengths
and the places where masks, pages and scales go wrong."""

import math

import numpy as np
import pytest
import torch

import oracle
from cache_util import Batch, check_attention, to_bf16
from exact_attention_fattn_gb300 import _lib
from exact_attention_fattn_gb300 import attention as A
from exact_attention_fattn_gb300 import cache as K

pytestmark = pytest.mark.gpu
C = oracle.cache


def status_ok():
    assert A.fattn_check_status() == 0


def run_attend(b, causal=True, selected=None, page_gap=0, scale=None, q=None, **kw):
    c, *where = b.device(page_gap)
    scale = A.default_scale(b.d) if scale is None else scale
    sel = None if selected is None else torch.from_numpy(selected).cuda()
    q = b.rows(b.q) if q is None else q
    out = torch.full((b.T, b.hq, b.d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.T, b.hq), 7.0, device="cuda")
    o, l = K.fattn_cache_fwd(q, c, *where, causal=causal, scale=scale, selected=sel, out=out, lse=lse, **kw)
    status_ok()
    return o.float().cpu().numpy().astype(np.float64), l.cpu().numpy().astype(np.float64)


def check(b, causal=True, selected=None, **kw):
    scale = A.default_scale(b.d)
    o, l = run_attend(b, causal, selected, **kw)
    want = C.attend(b.q, b.cache, b.table, b.q_start, b.kv_len, causal, scale, selected)
    kmax = 0.0
    for i, t in enumerate(b.lens):
        if t:
            kmax = max(kmax, float(np.nan_to_num(np.abs(C.cached_values(b.cache, b.table[i], t)[0])).max()))
    check_attention(o, l, want, b.d, float(np.abs(b.q).max()), kmax)
    behind = int(b.q_start[-1])
    assert (o[behind:] == 7.0).all() and (l[behind:] == 7.0).all()   # padding rows stay as they were
    return o, l, want


# ------------------------------------------------------------------ append

def run_append(b, rope_dim=0, interleaved=False, with_q=True, bounds=True, page_gap=0):
    c, *where = b.device(page_gap)
    if not bounds:
        c = c._replace(k_bounds=None)
    rope = K.fattn_rope_table(max(b.lens) + 3, rope_dim) if rope_dim else None
    fused = torch.cat([x.flatten(1) for x in (b.rows(b.q), b.rows(b.k_new), b.rows(b.v_new))], dim=1)
    nq, nk = b.hq * b.d, b.hkv * b.d
    q = fused[:, :nq].unflatten(1, (b.hq, b.d))
    k = fused[:, nq:nq + nk].unflatten(1, (b.hkv, b.d))
    v = fused[:, nq + nk:].unflatten(1, (b.hkv, b.d))
    q_out = torch.full((b.T, b.hq, b.d), 7.0, dtype=torch.bfloat16, device="cuda")
    got_q = K.fattn_cache_append(k, v, c, *where, rope=rope, q=q if with_q else None, interleaved=interleaved,
                                 q_out=q_out if with_q else None)
    status_ok()
    return c, got_q, None if rope is None else rope.cpu().numpy()


def check_append(b, rope_dim=0, interleaved=False, **kw):
    c, got_q, rope = run_append(b, rope_dim, interleaved, **kw)
    want = {k: v.copy() for k, v in b.cache.items()}
    if c.k_bounds is None:
        want["bounds"] = None
    q = C.append(want, b.k_new, b.v_new, b.table, b.q_start, b.kv_len, rope, interleaved, b.q)
    for name in ("k", "v", "k_scale", "v_scale"):
        assert np.array_equal(getattr(c, name).cpu().numpy(), want[name]), name
    if c.k_bounds is not None:
        assert np.array_equal(c.k_bounds.cpu().numpy(), want["bounds"])
    if got_q is not None:
        n = int(b.q_start[-1])
        assert np.array_equal(got_q.float().cpu().numpy()[:n], to_bf16(q[:n]))
        assert (got_q.float().cpu().numpy()[n:] == 7.0).all()
    return want


@pytest.mark.parametrize("d,page", [(64, 32), (64, 64), (64, 128), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("lens,news", [
    ([1], [1]), ([33, 128, 1, 65], [1, 1, 1, 1]), ([300, 129, 64], [300, 2, 64]), ([257, 31, 500], [130, 0, 77])])
def test_append(d, page, lens, news):
    b = Batch(sum(lens) + d + page, lens, news, 2, 3, d, page, pad_rows=3, filled=False)
    check_append(b, rope_dim=d, interleaved=bool(len(lens) & 1))


@pytest.mark.parametrize("rope_dim,interleaved", [(0, False), (16, False), (48, False), (112, True), (128, True), (32, True)])
def test_append_rotations(rope_dim, interleaved):
    check_append(Batch(3, [200, 77], [90, 5], 3, 5, 128, 64, filled=False), rope_dim, interleaved)


def test_append_without_queries_bounds_and_with_gaps():
    check_append(Batch(4, [100, 40], [50, 1], 2, 1, 64, 32, filled=False), 64, with_q=False)
    check_append(Batch(4, [100, 40], [50, 1], 2, 1, 64, 32, filled=False), 64, bounds=False)
    check_append(Batch(4, [100, 40], [50, 1], 2, 1, 64, 32, filled=False), 64, page_gap=48)


def test_append_many_sequences():
    """More sequences than one round of the warp's search (32) and two (1024)."""
    r = np.random.default_rng(1)
    for n in (33, 1030):
        lens = r.integers(1, 40, n).tolist()
        news = [int(r.integers(0, t + 1)) for t in lens]
        check_append(Batch(n, lens, news, 1, 1, 64, 32, pad_rows=2, filled=False), 64)


def test_append_grows_a_pages_scale():
    """Each token is larger than the last: every append raises the scale and
    rounds the page's codes again."""
    b = Batch(6, [40], [1], 2, 1, 64, 64, filled=False)
    c, table, _, _ = b.device()
    want = {k: v.copy() for k, v in b.cache.items()}
    qs = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for t in range(40):
        k = to_bf16(np.random.default_rng(t).standard_normal((1, 2, 64)) * 2.0 ** (t / 4 - 3))
        C.append(want, k, -k, b.table, np.array([0, 1]), np.array([t + 1]))
        K.fattn_cache_append(b.rows(k), b.rows(-k), c, table, qs, torch.tensor([t + 1], dtype=torch.int32, device="cuda"))
    status_ok()
    for name in ("k", "v", "k_scale", "v_scale"):
        assert np.array_equal(getattr(c, name).cpu().numpy(), want[name]), name
    assert np.array_equal(c.k_bounds.cpu().numpy(), want["bounds"])


def test_append_zeros_infinities_and_nan():
    b = Batch(8, [64, 64, 40], [64, 30, 40], 2, 1, 64, 32, filled=False)
    b.k_new[:70] = 0
    b.v_new[:64] = 0
    b.k_new[80, 0, 3] = np.inf
    b.v_new[81, 1, 5] = -np.inf
    b.k_new[100, 0, 7] = np.nan
    b.v_new[101, 1, 9] = np.nan
    b.v_new[94:134, 0] = np.nan     # a fresh page of NaN tokens alone (head 0, sequence 2)
    want = check_append(b)
    assert (want["k_scale"] == 2.0 ** 48).any() and (want["k_scale"] == 2.0 ** -48).any()


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("d,page", [(64, 32), (64, 64), (64, 128), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("g", [1, 4, 7, 16])
def test_attend_tokens(d, page, g):
    lens = [1, 31, 32, 33, 255, 256, 257, 600, 1029]
    check(Batch(d + page + g, lens, [1] * len(lens), 2, g, d, page, pad_rows=2))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,news,hkv,g", [
    ([300, 40, 500], [3, 2, 3], 2, 5), ([70, 700], [70, 1], 1, 3), ([513, 2, 100], [130, 2, 0], 3, 1),
    ([400], [150], 1, 12), ([130, 260], [129, 140], 2, 8)])
def test_attend_ragged(d, causal, lens, news, hkv, g):
    check(Batch(sum(lens) + d, lens, news, hkv, g, d, 64, pad_rows=1), causal)


@pytest.mark.parametrize("page", [32, 64, 128])
def test_attend_prompts(page):
    """Whole prompts and pieces of them, several row tiles each."""
    check(Batch(page, [300, 700, 1], [300, 200, 1], 1, 2, 128, page, pad_rows=5))
    check(Batch(page, [517], [517], 2, 1, 64, page))


def test_attend_long():
    """Many CTAs on one sequence: partial results joined over the whole grid."""
    check(Batch(21, [40000], [1], 1, 4, 128, 128))
    check(Batch(22, [30001, 5, 12000], [1, 1, 1], 2, 2, 64, 64))
    check(Batch(23, [9000, 777], [20, 9], 1, 8, 128, 64))


def test_attend_rows_that_see_nothing():
    """Empty sequences, and more new rows than cached tokens: the rows before
    position 0 see nothing."""
    check(Batch(31, [0, 5, 0, 130], [3, 9, 0, 1], 2, 2, 64, 32, pad_rows=2))
    check(Batch(32, [3, 0], [200, 2], 1, 4, 128, 64))
    check(Batch(32, [0, 0], [200, 2], 1, 4, 128, 64))


def test_attend_scale_extremes():
    """Pages whose value and key scales differ by 2^40, and the ends of the range."""
    for news in ([1, 1], [40, 33]):
        b = Batch(41, [300, 500], news, 1, 4, 128, 32, spread=0)
        r = np.random.default_rng(0)
        b.cache["v_scale"][:] = 2.0 ** r.integers(-20, 21, b.cache["v_scale"].shape)
        check(b)
        b.cache["v_scale"][:] = 2.0 ** 48
        b.cache["v_scale"][b.table[0, 0]] = 2.0 ** -48
        check(b)
        b.cache["v_scale"][:] = 2.0 ** -48
        check(b)


def test_attend_rows_of_one_page_of_small_values():
    """A row whose weight lies on a page with tiny values keeps their precision
    although other pages' values are 2^30 times larger."""
    for news in (1, 20):
        b = Batch(42, [256], [news], 1, 2, 128, 64, spread=0)
        b.cache["k"][:] = 0
        b.cache["k"][b.table[0, 1], 0, :, 0] = oracle.e4m3_encode(np.float32(448))
        b.q[:] = 0
        b.q[:, :, 0] = 64.0          # scores of the page: far above the others'
        b.cache["k_scale"][:] = 1.0
        b.cache["v_scale"][:] = 2.0 ** 20
        b.cache["v_scale"][b.table[0, 1]] = 2.0 ** -20
        o, l = run_attend(b)
        want = C.attend(b.q, b.cache, b.table, b.q_start, b.kv_len, True, A.default_scale(128))
        # scores of 2534 nats above the rest: exact zeros elsewhere, a plain
        # mean of the page's values (fp16 and bf16 rounding, A bounds the sum)
        allow = 2.0 ** -8 * np.abs(want[0]) + 2.0 ** -10 * want[2]
        assert (np.abs(o - want[0]) <= allow).all()


def test_attend_query_magnitudes():
    for mag in (2.0 ** -90, 2.0 ** -20, 2.0 ** 12):
        for news in ([1, 1], [30, 2]):
            b = Batch(43, [200, 70], news, 1, 4, 64, 32)
            b.q *= np.float32(mag)
            b.q[0] = 0
            scale = float(np.float32(0.125 / mag))
            o, l = run_attend(b, scale=scale)
            want = C.attend(b.q, b.cache, b.table, b.q_start, b.kv_len, True, scale)
            check_attention(o, l, want, 64, float(np.abs(b.q).max()) / mag, 448 * 2.0 ** -4)


@pytest.mark.parametrize("news", [1, 3, 40])
def test_nan_token_reaches_its_readers_only(news):
    """A NaN key (what append stores for a token with a NaN) gives NaN rows to
    those that attend to it, and leaves all others alone."""
    b = Batch(51, [150, 150], [news, news], 2, 2, 64, 32)
    at = 150 - 1 - news // 2         # visible to the later new rows only
    b.cache["k"][b.table[0, at // 32], 1, at % 32, 5] = 0x7F
    o, l = run_attend(b)
    want = C.attend(b.q, b.cache, b.table, b.q_start, b.kv_len, True, A.default_scale(64))
    assert np.array_equal(np.isnan(o), np.isnan(want[0])) and np.array_equal(np.isnan(l), np.isnan(want[1]))
    assert np.isnan(o).any()
    check_attention(o, l, want, 64, float(np.abs(b.q).max()), 448 * 2.0 ** -4)   # the other rows


def test_attend_strided_rows_and_pages():
    b = Batch(61, [200, 90], [2, 1], 2, 4, 128, 64)
    wide = torch.full((b.T, 3 * b.hq * b.d), float("nan"), dtype=torch.bfloat16, device="cuda")
    q = wide[:, b.hq * b.d:2 * b.hq * b.d].unflatten(1, (b.hq, b.d))
    q.copy_(b.rows(b.q))
    check(b, page_gap=64, q=q)
    b = Batch(62, [200, 190], [100, 30], 2, 4, 128, 64)
    check(b, page_gap=16)


def test_pages_shared_between_sequences():
    """Two sequences on the same pages (a shared prompt)."""
    b = Batch(63, [250, 128], [1, 1], 1, 4, 64, 64)
    b.table[1, :2] = b.table[0, :2]
    check(b)


def test_pages_beyond_32_bit_offsets():
    """Codes more than 2^32 bytes into the cache."""
    pages, hkv, page, d = 70000, 8, 64, 128
    for news in ([1, 1], [70, 3]):
        b = Batch(64, [150, 64], news, hkv, 2, d, page)
        c0, table, qs, kl = b.device()
        big = K.fattn_cache_alloc(pages, hkv, d, page, bounds=True)
        move = pages - b.pages
        for x, y in zip(big, c0):
            x[move:] = y
        table2 = torch.where(table < b.pages, table + move, table)
        q = b.rows(b.q)
        o, l = K.fattn_cache_fwd(q, big, table2, qs, kl)
        o0, l0 = K.fattn_cache_fwd(q, c0, table, qs, kl)
        k, v = b.rows(b.k_new), b.rows(b.v_new)
        K.fattn_cache_append(k, v, big, table2, qs, kl)
        K.fattn_cache_append(k, v, c0, table, qs, kl)
        s = K.fattn_cache_select(q, big, table2, qs, kl, 1)
        s0 = K.fattn_cache_select(q, c0, table, qs, kl, 1)
        status_ok()
        assert torch.equal(o, o0) and torch.equal(l, l0) and torch.equal(s, s0)
        for x, y in zip(big, c0):
            assert torch.equal(x[move:].view(torch.uint8), y.view(torch.uint8))
        del big
        torch.cuda.empty_cache()


# ------------------------------------------------------------------ selection

def run_select(b, k, first, recent):
    c, *where = b.device()
    out = torch.full((b.T, b.hkv, k), -2, dtype=torch.int32, device="cuda")
    s = K.fattn_cache_select(b.rows(b.q), c, *where, k, n_first=first, n_recent=recent, out=out)
    status_ok()
    return s.cpu().numpy()


@pytest.mark.parametrize("d,page", [(64, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("g,k,first,recent", [(1, 1, 0, 0), (3, 5, 1, 2), (8, 16, 0, 1), (128, 4, 2, 2)])
def test_select(d, page, g, k, first, recent):
    b = Batch(d + page + g, [page * 40 + 3, 1, 0, page * 4, page * 300], [2, 1, 1, 0, 1], 2, g, d, page, pad_rows=2)
    want = C.select(b.q, b.cache, b.table, b.q_start, b.kv_len, k, first, recent)
    assert np.array_equal(run_select(b, k, first, recent), want)


def test_select_ties_go_to_the_lower_page():
    b = Batch(71, [32 * 600], [1], 2, 2, 64, 32)
    b.cache["bounds"][:] = b.cache["bounds"][0]
    b.cache["k_scale"][:] = 1.0
    want = C.select(b.q, b.cache, b.table, b.q_start, b.kv_len, 20, 0, 1)
    assert want[0, 0].tolist() == list(range(19)) + [599]
    assert np.array_equal(run_select(b, 20, 0, 1), want)
    b.q[:] = 0                       # nothing scores
    b.q[0, 0, 0] = 2.0 ** -110
    assert np.array_equal(run_select(b, 20, 0, 1), want)


@pytest.mark.parametrize("d,page,g,k", [(128, 64, 4, 8), (64, 32, 1, 3), (128, 128, 20, 5), (64, 64, 16, 40)])
def test_attend_selected(d, page, g, k):
    b = Batch(81 + d, [page * 30 + 5, 3, page * 11, 0], [1, 1, 3, 1], 2, g, d, page, pad_rows=2)
    sel = C.select(b.q, b.cache, b.table, b.q_start, b.kv_len, k, 1, 1)
    check(b, selected=sel)
    sel[0, 0, :] = -1                # a row with nothing selected
    check(b, selected=sel)
    sel[0, 1, 0] = 1 << 20           # rows that no page table has are reported, not read
    b.table[:] = np.where(b.table >= b.pages, 0, b.table)
    c, *where = b.device()
    K.fattn_cache_fwd(b.rows(b.q), c, *where, selected=torch.from_numpy(sel).cuda())
    assert A.fattn_check_status() == _lib.FATTN_ERR_BAD_INDEX


def test_selected_twice_counts_twice():
    b = Batch(83, [500], [1], 1, 2, 64, 64)
    once = np.array([[[1, 2]]], dtype=np.int32)
    twice = np.array([[[1, 1, 2, 2]]], dtype=np.int32)
    o1, l1 = run_attend(b, selected=once)
    o2, l2 = run_attend(b, selected=twice)
    assert np.abs(o1 - o2).max() <= 2.0 ** -7 * np.abs(o1).max()
    assert np.abs(l2 - l1 - math.log(2.0)).max() < 1e-5


# ------------------------------------------------------------------ checks on the device

@pytest.mark.parametrize("what", ["page", "negative page", "q_start", "kv_len", "negative kv_len"])
@pytest.mark.parametrize("news", [1, 50])
def test_bad_indices_are_reported_not_followed(what, news):
    b = Batch(91, [200, 100], [news, news], 1, 2, 64, 32)
    if what == "page":
        b.table[0, 2] = b.pages
    elif what == "negative page":
        b.table[0, 2] = -5
    elif what == "q_start":
        b.q_start = np.array([0, 3 * news, 2 * news], dtype=np.int32)
    elif what == "kv_len":
        b.kv_len[0] = b.max_pages * 32 + 1
    else:
        b.kv_len[0] = -1
    c, *where = b.device()
    q = b.rows(b.q)
    sel = torch.zeros((b.T, 1, 8), dtype=torch.int32, device="cuda") + torch.arange(8, device="cuda", dtype=torch.int32)
    calls = [lambda: K.fattn_cache_fwd(q, c, *where), lambda: K.fattn_cache_fwd(q, c, *where, selected=sel),
             lambda: K.fattn_cache_select(q, c, *where, 2)]
    if "page" not in what:
        calls.append(lambda: K.fattn_cache_append(b.rows(b.k_new), b.rows(b.v_new), c, *where))
    for call in calls:
        call()
        assert A.fattn_check_status() == _lib.FATTN_ERR_BAD_INDEX
        status_ok()


def test_append_reports_bad_pages_and_positions():
    b = Batch(92, [200, 100], [1, 50], 1, 2, 64, 32, filled=False)
    b.table[1, 2] = b.pages + 7
    c, *where = b.device()
    before = c.k.clone()
    K.fattn_cache_append(b.rows(b.k_new), b.rows(b.v_new), c, *where)
    assert A.fattn_check_status() == _lib.FATTN_ERR_BAD_INDEX
    assert not torch.equal(before, c.k)      # the other pages were served
    b = Batch(92, [200, 100], [1, 50], 1, 2, 64, 32, filled=False)
    c, *where = b.device()
    rope = K.fattn_rope_table(150, 64)       # sequence 0's token lies behind it
    K.fattn_cache_append(b.rows(b.k_new), b.rows(b.v_new), c, *where, rope=rope, q=b.rows(b.q))
    assert A.fattn_check_status() == _lib.FATTN_ERR_BAD_INDEX
    status_ok()


def test_binding_refuses():
    b = Batch(93, [64], [1], 2, 2, 64, 32)
    c, table, qs, kl = b.device()
    q = b.rows(b.q)
    good = (q, c, table, qs, kl)
    for i, bad in ((0, q.float()), (0, q.cpu()), (0, q[:, :, :32]), (0, q.transpose(1, 2)), (2, table.long()),
                   (2, table.cpu()), (3, qs[:1]), (4, kl.view(1, 1)), (1, c._replace(k=c.k.float())),
                   (1, c._replace(v=c.v[:1])), (1, c._replace(k_scale=c.k_scale.double())),
                   (1, c._replace(k=c.k.transpose(2, 3)))):
        args = list(good)
        args[i] = bad
        with pytest.raises((TypeError, ValueError)):
            K.fattn_cache_fwd(*args)
    with pytest.raises(ValueError):
        K.fattn_cache_fwd(*good, out=torch.empty_like(q, dtype=torch.float32))
    with pytest.raises(_lib.FattnError):
        K.fattn_cache_fwd(*good, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(_lib.FattnError):
        K.fattn_cache_fwd(*good, scale=-1.0)
    with pytest.raises(ValueError):
        K.fattn_cache_select(q, c._replace(k_bounds=None), table, qs, kl, 2)
    with pytest.raises(_lib.FattnError):
        K.fattn_cache_select(*good, 2, n_first=2, n_recent=1)
    with pytest.raises(ValueError):
        K.fattn_cache_append(q[:, :1], q[:, :2], *good[1:])
    with pytest.raises(ValueError):          # three query heads over two kv heads
        K.fattn_cache_fwd(q[:, :3].contiguous(), *good[1:])
    status_ok()


# ------------------------------------------------------------------ as they are used

def test_serving_loop():
    """Prompts, then tokens one by one: append, attend, select and attend to
    the selection, against the oracle's cache at every step."""
    hkv, g, d, page = 2, 3, 64, 32
    b = Batch(101, [150, 61, 90], [150, 61, 90], hkv, g, d, page)
    b.table = np.array([[*np.random.default_rng(i).permutation(5) * 3 + i, 99] for i in range(3)], dtype=np.int32)
    cache = K.fattn_cache_alloc(15, hkv, d, page, bounds=True)
    want = {"k": cache.k.cpu().numpy(), "v": cache.v.cpu().numpy(), "k_scale": cache.k_scale.cpu().numpy(),
            "v_scale": cache.v_scale.cpu().numpy(), "bounds": cache.k_bounds.cpu().numpy()}
    table = torch.from_numpy(b.table).cuda()
    rope = K.fattn_rope_table(200, d)
    r = np.random.default_rng(0)
    lens = np.zeros(3, dtype=np.int32)
    for step, news in enumerate([[150, 61, 90], [1, 1, 1], [1, 0, 1], [4, 3, 2], [1, 1, 1], [1, 33, 1]]):
        lens = lens + np.array(news, dtype=np.int32)
        qs = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        q, k, v = (to_bf16(r.standard_normal((qs[-1], h, d))) for h in (hkv * g, hkv, hkv))
        where = (table, torch.from_numpy(qs).cuda(), torch.from_numpy(lens).cuda())
        qr = K.fattn_cache_append(b.rows(k), b.rows(v), cache, *where, rope=rope, q=b.rows(q))
        q_ref = to_bf16(C.append(want, k, v, b.table, qs, lens, rope.cpu().numpy(), False, q))
        assert np.array_equal(qr.float().cpu().numpy(), q_ref)
        assert np.array_equal(cache.k.cpu().numpy(), want["k"]) and np.array_equal(cache.k_bounds.cpu().numpy(), want["bounds"])
        scale = A.default_scale(d)
        o, l = K.fattn_cache_fwd(qr, cache, *where)
        kmax = float(np.abs(oracle.e4m3_decode(want["k"]) * want["k_scale"][:, :, None, None]).max())
        check_attention(o.double().cpu().numpy(), l.double().cpu().numpy(),
                        C.attend(q_ref, want, b.table, qs, lens, True, scale), d, float(np.abs(q_ref).max()), kmax)
        sel = K.fattn_cache_select(qr, cache, *where, 3, n_first=1, n_recent=1)
        sel_ref = C.select(q_ref, want, b.table, qs, lens, 3, 1, 1)
        assert np.array_equal(sel.cpu().numpy(), sel_ref)
        o, l = K.fattn_cache_fwd(qr, cache, *where, selected=sel)
        check_attention(o.double().cpu().numpy(), l.double().cpu().numpy(),
                        C.attend(q_ref, want, b.table, qs, lens, True, scale, sel_ref), d,
                        float(np.abs(q_ref).max()), kmax)
    status_ok()


def test_results_repeat_bit_for_bit():
    b = Batch(111, [5000, 700, 1300], [1, 1, 1], 2, 4, 128, 64)
    c, *where = b.device()
    q = b.rows(b.q)
    first = K.fattn_cache_fwd(q, c, *where)
    for _ in range(5):
        again = K.fattn_cache_fwd(q, c, *where)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    status_ok()


@pytest.mark.parametrize("news", [1, 60])
def test_captured_and_replayed_with_other_lengths(news):
    """A captured step reads lengths, tables and pages when it runs."""
    b1 = Batch(121, [900, 300], [news, news], 1, 4, 128, 64, spare=20)
    b2 = Batch(122, [130, 1000], [news, news], 1, 4, 128, 64, spare=20)
    pages = max(b1.pages, b2.pages)
    static = K.fattn_cache_alloc(pages, 1, 128, 64, bounds=True)
    table = torch.zeros((2, 17), dtype=torch.int32, device="cuda")
    qs, kl = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (3, 2))
    q = torch.zeros((b1.T, 4, 128), dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros((b1.T, 1, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def load(b):
        c, t, s, l = b.device()
        for x, y in zip(static, c):
            x[:b.pages].copy_(y)
        table[:, :t.shape[1]].copy_(t)
        qs.copy_(s)
        kl.copy_(l)
        q.copy_(b.rows(b.q))
        k.copy_(b.rows(b.k_new))
        v.copy_(b.rows(b.v_new))

    def step():
        K.fattn_cache_append(k, v, static, table, qs, kl)
        sel = K.fattn_cache_select(q, static, table, qs, kl, 3)
        return (*K.fattn_cache_fwd(q, static, table, qs, kl), *K.fattn_cache_fwd(q, static, table, qs, kl, selected=sel))

    load(b1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for b in (b2, b1):
        load(b)
        g.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in out]
        load(b)
        for x, y in zip(got, step()):
            assert torch.equal(x, y)
    status_ok()


def test_two_streams_at_once():
    """Calls on two streams, each with its workspace."""
    bs = [Batch(131 + i, [3000, 200], [1, 1], 2, 4, 128, 64) for i in range(2)]
    dev = [b.device() for b in bs]
    qs = [b.rows(b.q) for b in bs]
    want = [K.fattn_cache_fwd(q, *d) for q, d in zip(qs, dev)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in bs]
    for _ in range(20):
        got = []
        for s, q, d in zip(streams, qs, dev):
            with torch.cuda.stream(s):
                got.append(K.fattn_cache_fwd(q, *d))
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    status_ok()


# ------------------------------------------------------------------ sizes at the kernels' edges

@pytest.mark.parametrize("d,page", [(64, 32), (64, 128), (128, 32), (128, 64), (128, 128)])
def test_attend_row_counts_around_the_tiles(d, page):
    """Units of 65 to 300 rows on one key tile to four, whole and shared
    between CTAs, beside a single token."""
    check(Batch(141, [65, 256, 134, 257, 1, 500, 300, 128, 390], [65, 128, 129, 255, 1, 257, 300, 127, 66], 2, 1, d, page))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g,news", [(12, [7, 6, 11]), (5, [40, 52, 26]), (33, [4, 3, 9])])
def test_attend_groups_that_split_tiles_unevenly(d, g, news):
    """Rows of one token on both sides of a tile's end."""
    check(Batch(142, [900, 131, 513], news, 1, g, d, 64))


@pytest.mark.parametrize("news,g", [(1, 2), (5, 16)])
def test_attend_most_sequences(news, g):
    """4096 sequences of a few tokens, some without rows."""
    r = np.random.default_rng(143)
    lens = [int(x) for x in r.integers(news, 40, 4096)]
    check(Batch(143, lens, [news if i % 7 else 0 for i in range(4096)], 1, g, 128, 32, pad_rows=3))


@pytest.mark.parametrize("seed", range(16))
def test_attend_drawn_batches(seed):
    r = np.random.default_rng(1000 + seed)
    d, page, g, hkv = (int(r.choice(x)) for x in ([64, 128], [32, 64, 128], [1, 2, 3, 5, 8, 16], [1, 2, 3]))
    B = int(r.integers(1, 9))
    most = int(r.choice([1, 4, 30, 200]))
    lens = [int(x) for x in np.exp(r.uniform(0, np.log(3000), B)).astype(int) + 1]
    news = [min(t, int(r.integers(0, most + 1))) for t in lens]
    news[0] = max(1, news[0])
    check(Batch(150 + seed, lens, news, hkv, g, d, page, pad_rows=seed % 3), causal=seed % 5 != 0)


@pytest.mark.parametrize("lens,news,hkv,k", [
    ([2300 * 32], [2], 1, 20),                      # eight CTAs a pair
    ([2300 * 32 - 5, 70], [70, 2], 1, 20),          # four, and pairs with fewer pages than the CTAs start at
    ([2300 * 32 - 5, 70], [80, 2], 2, 20),          # one
    ([500 * 32 - 3, 9000], [30, 150], 2, 20),       # small CTAs, pages in several turns
    ([10400 * 32 - 31], [80], 2, 40)])              # scores in the workspace: more pages than fit
def test_select_many_pages(lens, news, hkv, k):
    b = Batch(144, lens, news, hkv, 2, 64, 32)
    assert np.array_equal(run_select(b, k, 1, 2), C.select(b.q, b.cache, b.table, b.q_start, b.kv_len, k, 1, 2))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("news", [[1, 1], [3, 0], [2, 70]])
def test_largest_group(d, news):
    """128 query heads share a kv head: one token's rows are eight small units or
    half a large one."""
    b = Batch(181, [300, 129], news, 1, 128, d, 64, pad_rows=1)
    check(b)
    sel = np.full((b.T, 1, 3), -1, np.int32)
    sel[:, 0, 0], sel[:, 0, 2] = 1, 0
    check(b, selected=sel)


@pytest.mark.parametrize("news", [[1, 1], [30, 2]])
def test_most_kv_heads(news):
    b = Batch(182, [70, 33], news, 1024, 1, 64, 32)
    check(b)
    check_append(Batch(183, [70, 33], news, 1024, 1, 64, 32, filled=False))
    assert np.array_equal(run_select(b, 2, 0, 1), C.select(b.q, b.cache, b.table, b.q_start, b.kv_len, 2, 0, 1))


@pytest.mark.parametrize("causal", [True, False])
def test_one_token_cached(causal):
    for d, page in ((64, 32), (128, 128)):
        check(Batch(184, [1], [1], 1, 1, d, page), causal)
        check(Batch(185, [1, 2, 1], [0, 2, 1], 2, 40, d, page), causal)


def test_strided_queries_and_pages_for_many_rows():
    """Rows cut out of one projection, pages apart, 300 rows a sequence."""
    b = Batch(186, [700, 310], [300, 310], 2, 2, 128, 64, pad_rows=3)
    wide = torch.full((b.T, b.hq * b.d + 64), 9.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :b.hq * b.d] = b.rows(b.q).flatten(1)
    check(b, page_gap=48, q=wide[:, :b.hq * b.d].unflatten(1, (b.hq, b.d)))


@pytest.mark.parametrize("news", [[1, 2], [40, 300]])
@pytest.mark.parametrize("d", [64, 128])
def test_outputs_on_a_16_byte_boundary(news, d):
    b = Batch(187, [700, 310], news, 2, 2, d, 64)
    c, *where = b.device()
    q = b.rows(b.q)
    buf = torch.full((q.numel() + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[8:8 + q.numel()].view(q.shape)
    assert out.data_ptr() % 32 == 16
    o, lse = K.fattn_cache_fwd(q, c, *where)
    o2, lse2 = K.fattn_cache_fwd(q, c, *where, out=out)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert bool((buf[:8] == 7.0).all()) and bool((buf[8 + q.numel():] == 7.0).all())
    status_ok()


# ------------------------------------------------------------------ memory the caller owns

def test_queries_rotated_in_place():
    b = Batch(145, [150, 40], [60, 1], 2, 4, 128, 64, pad_rows=2, filled=False)
    c, *where = b.device()
    rope = K.fattn_rope_table(150, 96)
    q = b.rows(b.q)
    want = K.fattn_cache_append(b.rows(b.k_new), b.rows(b.v_new), c, *where, rope=rope, q=q)[:61].clone()
    got = K.fattn_cache_append(b.rows(b.k_new), b.rows(b.v_new), c, *where, rope=rope, q=q, q_out=q)
    assert got is q and torch.equal(q[:61], want) and torch.equal(q[61:], b.rows(b.q)[61:])
    status_ok()


def test_one_workspace_of_the_stated_size_for_call_after_call():
    """Whatever the last call left in it; nothing behind it is written."""
    bs = [Batch(146, [900, 131], [1, 1], 2, 4, 128, 64), Batch(147, [900, 500], [90, 200], 2, 4, 128, 64),
          Batch(148, [700, 64], [3, 2], 2, 16, 64, 32)]
    ws = None
    for b in bs * 2:
        c, *where = b.device()
        q = b.rows(b.q)
        sel = K.fattn_cache_select(q, c, *where, 4)
        for s in (None, sel):
            need = K.fattn_cache_fwd_workspace_bytes(b.T, 2, b.hq, 2, b.d, 0 if s is None else 4)
            if ws is None:
                ws = torch.full((1 << 27,), 0xFF, dtype=torch.uint8, device="cuda")
            assert need < ws.numel()
            ws[need:need + 4096] = 0xA5
            got = K.fattn_cache_fwd(q, c, *where, selected=s, workspace=ws[:need])
            want = K.fattn_cache_fwd(q, c, *where, selected=s)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            assert bool((ws[need:need + 4096] == 0xA5).all())
    status_ok()


def test_streams_and_graphs_at_once():
    """Both attention kernels, the selection and a replayed graph on four
    streams; every call has its own workspace."""
    bs = [Batch(161, [3000, 200], [1, 1], 2, 4, 128, 64), Batch(162, [2000, 700], [300, 90], 2, 4, 128, 64),
          Batch(163, [4000, 900], [2, 1], 2, 4, 64, 32), Batch(164, [1500, 1100], [70, 250], 2, 4, 64, 128)]
    dev = [b.device() for b in bs]
    qs = [b.rows(b.q) for b in bs]

    def call(i):
        q, d = qs[i], dev[i]
        sel = K.fattn_cache_select(q, *d, 5) if i == 2 else None
        return K.fattn_cache_fwd(q, *d, selected=sel)

    want = [tuple(x.clone() for x in call(i)) for i in range(4)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out3 = call(3)
    streams = [torch.cuda.Stream() for _ in bs]
    for _ in range(20):
        got = [None] * 4
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                if i == 3:
                    graph.replay()
                    got[3] = out3
                else:
                    got[i] = call(i)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    status_ok()


@pytest.mark.parametrize("news", [3, 90])
def test_overlapping_sequences_are_reported(news):
    """q_start that goes back: the sequence between is empty, and reported."""
    b = Batch(149, [200, 150, 180], [news, 0, 0], 1, 2, 64, 32)
    b.q_start = np.array([0, news, 0, news], dtype=np.int32)
    c, *where = b.device()
    K.fattn_cache_fwd(b.rows(b.q), c, *where)
    assert A.fattn_check_status() == _lib.FATTN_ERR_BAD_INDEX
    status_ok()
