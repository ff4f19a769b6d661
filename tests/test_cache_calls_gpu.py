"""Calls of the paged cache's entry points as programs make them beyond the
plain ones of test_cache_gpu.py: from several threads, with batches that are
partly senseless, with infinities among the queries."""

import threading

import numpy as np
import pytest
import torch

import oracle
from cache_util import Batch, to_bf16
from exact_attention_fattn_gb300 import _lib
from exact_attention_fattn_gb300 import attention as A
from exact_attention_fattn_gb300 import cache as K

pytestmark = pytest.mark.gpu
C = oracle.cache


def test_threads_with_batches_of_different_sizes():
    """Eight host threads, a stream each; the batches, and with them the
    shared memory that a call asks for, differ."""
    bs = [Batch(300 + i, [3 + i] * n, [new] * n, 1, 2, 64 if i & 1 else 128, 32)
          for i, (n, new) in enumerate([(1, 1), (900, 1), (40, 1), (1500, 1), (1, 40), (30, 50), (3, 60), (70, 45)])]
    dev = [b.device() for b in bs]
    qs = [b.rows(b.q) for b in bs]
    torch.cuda.synchronize()
    got, errors = [None] * len(bs), []
    gate = threading.Barrier(len(bs))

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                gate.wait()
                for _ in range(20):
                    got[i] = K.fattn_cache_fwd(qs[i], *dev[i])
                torch.cuda.current_stream().synchronize()
        except Exception as e:
            errors.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(bs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert A.fattn_check_status() == 0
    for i, b in enumerate(bs):
        want = K.fattn_cache_fwd(qs[i], *dev[i])
        assert torch.equal(got[i][0], want[0]) and torch.equal(got[i][1], want[1])
    assert A.fattn_check_status() == 0


@pytest.mark.parametrize("news", [1, 60])
def test_host_path_on_public_functions_alone(news, monkeypatch):
    b = Batch(310, [500, 90], [news, news], 2, 2, 128, 64)
    d, q = b.device(), b.rows(b.q)
    want = K.fattn_cache_fwd(q, *d)
    monkeypatch.setattr(K, "_current_device", torch.cuda.current_device)
    monkeypatch.setattr(K, "_raw_stream", K._public_stream)
    monkeypatch.setattr(K, "_raw_alloc", None)
    for s in (torch.cuda.current_stream(), torch.cuda.Stream()):
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            got = K.fattn_cache_fwd(q, *d)
        s.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert A.fattn_check_status() == 0


@pytest.mark.parametrize("what", ["longer than its table", "negative length", "more new than cached",
                                  "past the rotation's table", "q_start past the rows"])
@pytest.mark.parametrize("rope_dim", [0, 64])
def test_append_leaves_out_the_queries_of_senseless_sequences(what, rope_dim):
    """A sequence whose keys are not appended has its rows of q_out left alone,
    too, and the other sequences are served."""
    if what == "past the rotation's table" and rope_dim == 0:
        pytest.skip("no rotation, no table")
    b = Batch(320, [60, 90, 40], [5, 40, 3], 2, 2, 64, 32, filled=False)
    c, table, qs, kl = b.device()
    rope, bad = None, 1
    if rope_dim:
        rope = K.fattn_rope_table(70 if what == "past the rotation's table" else 400, rope_dim)
    if what == "longer than its table":
        kl[1] = b.max_pages * 32 + 1
    elif what == "negative length":
        kl[1] = -1
    elif what == "more new than cached":
        kl[1] = 39                    # rows of positions -1 .. 38
    elif what == "q_start past the rows":
        bad = 2
        qs[3] = b.T + 1
    before = [x.clone() for x in c]
    q_out = torch.full((b.T, b.hq, b.d), 7.0, dtype=torch.bfloat16, device="cuda")
    K.fattn_cache_append(b.rows(b.k_new), b.rows(b.v_new), c, table, qs, kl, rope=rope, q=b.rows(b.q), q_out=q_out)
    assert A.fattn_check_status() == _lib.FATTN_ERR_BAD_INDEX
    rows = slice(int(b.q_start[bad]), int(b.q_start[bad + 1]))
    pages = table[bad, :-(-b.lens[bad] // 32)].long()
    assert all(torch.equal(x[pages], y[pages]) for x, y in zip(c, before))
    assert bool((q_out[rows] == 7.0).all())
    # the others: as without that sequence
    b.q_start = np.concatenate([[0], np.cumsum([n if i != bad else 0 for i, n in enumerate(b.news)])]).astype(np.int32)
    keep = np.ones(b.T, bool)
    keep[rows] = False
    want = {k: v.copy() for k, v in b.cache.items()}
    q = C.append(want, b.k_new[keep], b.v_new[keep], b.table, b.q_start, b.kv_len,
                 None if rope is None else rope.cpu().numpy(), False, b.q[keep])
    for name in ("k", "v", "k_scale", "v_scale"):
        assert np.array_equal(getattr(c, name).cpu().numpy(), want[name]), name
    assert np.array_equal(c.k_bounds.cpu().numpy(), want["bounds"])
    assert np.array_equal(q_out.float().cpu().numpy()[keep], to_bf16(q))
    assert A.fattn_check_status() == 0


@pytest.mark.parametrize("call", ["append", "append with queries", "attend", "attend selected", "select"])
@pytest.mark.parametrize("starts", [[0, 100, 0, 100], [0, 60, 40, 100], "long"])
def test_starts_that_go_back_are_reported(call, starts):
    """A sequence whose rows end before they begin is found by no search for a
    row or a page; rows of its neighbours may then belong to none."""
    if starts == "long":
        b = Batch(330, [600] * 600, [1] * 600, 1, 1, 64, 128)
        b.q_start[500] = 0
    else:
        b = Batch(331, [120, 130, 140], [100, 0, 0], 1, 2, 64, 32)
        b.q_start = np.array(starts, dtype=np.int32)
    c, *where = b.device()
    q = b.rows(b.q)
    if call.startswith("append"):
        K.fattn_cache_append(b.rows(b.k_new), b.rows(b.v_new), c, *where, q=q if "queries" in call else None)
    elif call == "attend":
        K.fattn_cache_fwd(q, c, *where)
    elif call == "select":
        K.fattn_cache_select(q, c, *where, 2)
    else:
        sel = torch.zeros((b.T, 1, 1), dtype=torch.int32, device="cuda")
        K.fattn_cache_fwd(q, c, *where, selected=sel)
    assert A.fattn_check_status() == _lib.FATTN_ERR_BAD_INDEX
    assert A.fattn_check_status() == 0


@pytest.mark.parametrize("B,T", [(600, 1), (4096, 3), (40, 700)])
def test_good_starts_are_not_reported(B, T):
    """Most sequences without rows, rows in front of the first and behind the last."""
    news = [0] * B
    news[B // 2] = T
    b = Batch(332, [900 if n else 40 for n in news], news, 1, 1, 64, 128, pad_rows=2)
    c, *where = b.device()
    sel = K.fattn_cache_select(b.rows(b.q), c, *where, 2)
    K.fattn_cache_fwd(b.rows(b.q), c, *where, selected=sel)
    K.fattn_cache_append(b.rows(b.k_new), b.rows(b.v_new), c, *where)
    assert A.fattn_check_status() == 0


@pytest.mark.parametrize("news", [1, 3, 40])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_infinite_queries(news, d, bad):
    """A query with an infinity has infinite scores and so a NaN row, also
    where all of them are -inf; it is no row that sees nothing.  Other rows
    and, in a group, other heads are as they were."""
    b = Batch(340, [150, 70], [news, news], 1, 3, d, 32)
    for p in b.table[:, :5].ravel():
        if p < b.pages:               # one sign in column 9: every score is -inf, or every one inf
            x = b.cache["k"][p, 0, :, 9]
            b.cache["k"][p, 0, :, 9] = np.where(x & 0x7F == 0x7F, x, (x & 0x7F) | 0x80 | 1)
    clean = b.device()
    o0, l0 = K.fattn_cache_fwd(b.rows(b.q), *clean)
    row = news // 2
    b.q[row, 1, 9] = bad
    sel = torch.zeros((b.T, 1, 1), dtype=torch.int32, device="cuda")
    for kw in ({}, {"causal": False}, {"selected": sel}):
        o, l = K.fattn_cache_fwd(b.rows(b.q), *clean, **kw)
        assert bool(torch.isnan(o[row, 1]).all()) and bool(torch.isnan(l[row, 1])), kw
        if kw == {}:
            keep = torch.ones((b.T, 3), dtype=torch.bool, device="cuda")
            keep[row, 1] = False
            assert torch.equal(o[keep], o0[keep]) and torch.equal(l[keep], l0[keep])
        else:
            assert int(torch.isnan(l).sum()) == 1
    assert A.fattn_check_status() == 0


@pytest.mark.parametrize("news", [1, 60])
@pytest.mark.parametrize("d", [64, 128])
def test_a_wait_budget_that_runs_out(news, d):
    """Waits that give up are reported, and the next call, on the same memory
    and on tensor memory that the last one handed back, is right."""
    b = Batch(350, [3000, 700], [news, news], 2, 2, d, 64)
    where, q = b.device(), b.rows(b.q)
    want = K.fattn_cache_fwd(q, *where)
    assert A.fattn_check_status() == 0
    A.fattn_set_wait_budget(1)
    try:
        for _ in range(3):
            K.fattn_cache_fwd(q, *where)
            assert A.fattn_check_status() in (_lib.FATTN_OK, _lib.FATTN_ERR_TIMEOUT)
    finally:
        A.fattn_set_wait_budget(0)
    for _ in range(3):
        got = K.fattn_cache_fwd(q, *where)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert A.fattn_check_status() == 0
