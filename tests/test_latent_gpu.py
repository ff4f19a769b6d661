"""The paged latent cache on the GPU: appending bit for bit against the oracle,
attention within bounds derived from the arithmetic (latent_util.check_latent),
over head counts, ranks, page sizes, ragged lengths and the places where masks
and pages go wrong."""

import numpy as np
import pytest
import torch

import exact_attention_fattn_gb300 as F
import oracle
from exact_attention_fattn_gb300 import _lib
from latent_util import ROPE, LatentBatch, check_latent

pytestmark = pytest.mark.gpu
C = oracle.latent


def ok():
    assert F.fattn_check_status() == 0


def arrays(o, lse):
    return o.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)


def run(b, causal=True, gap=0, scale=0.07, q=None, **kw):
    c, *where = b.device(gap)
    out = torch.full((b.T, b.heads, b.rank), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.T, b.heads), 7.0, device="cuda")
    F.fattn_latent_fwd(b.rows(b.q) if q is None else q, c, *where, scale=scale, causal=causal, out=out, lse=lse, **kw)
    ok()
    return arrays(out, lse)


def check(b, causal=True, scale=0.07, **kw):
    want = C.attend(b.q, b.data, b.rank, b.table, b.q_start, b.kv_len, causal, scale)
    behind = int(b.q_start[-1])
    for x in b.tables():
        o, l = run(x, causal, scale=scale, **kw)
        check_latent(o, l, want, b.rank + ROPE)
        assert (o[behind:] == 7.0).all() and (l[behind:] == 7.0).all()   # padding rows stay as they were
    return o, l, want


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("rank,page", [(256, 32), (256, 64), (256, 128), (512, 32), (512, 64), (512, 128)])
@pytest.mark.parametrize("heads", [1, 16, 20, 33, 64])
def test_single_tokens(rank, page, heads):
    """Sequences of one token up to a few tiles, ends inside pages and tiles."""
    check(LatentBatch(heads + page, [1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300, 2], [1] * 12, heads, rank, page, pad_rows=2))


@pytest.mark.parametrize("rank,page", [(256, 64), (512, 32), (512, 128)])
@pytest.mark.parametrize("heads,news", [(16, 5), (128, 1), (128, 3), (40, 2), (96, 1), (5, 30), (1, 200), (200, 1)])
def test_more_rows_than_a_block(rank, page, heads, news):
    """Row blocks side by side, the last of them partly filled, some without rows."""
    b = LatentBatch(heads * news, [news, 260, 515, news + 1, 700], [news, news, 1, 0, news], heads, rank, page, pad_rows=1)
    check(b)
    check(b, causal=False)


@pytest.mark.parametrize("rank", [256, 512])
@pytest.mark.parametrize("lens,news,heads", [([700], [700], 16), ([300, 90], [300, 33], 20), ([1200], [150], 64), ([64], [64], 128)])
def test_prompts(rank, lens, news, heads):
    """Whole prompts and pieces: masks on the diagonal, groups of up to eight blocks."""
    b = LatentBatch(sum(lens) + heads, lens, news, heads, rank, 64, pad_rows=1)
    check(b)
    if heads == 20:
        check(b, causal=False)


@pytest.mark.parametrize("rank,heads", [(512, 16), (512, 128), (256, 40)])
def test_long_sequences_shared_by_many_ctas(rank, heads):
    check(LatentBatch(heads, [12001], [1], heads, rank, 64))
    check(LatentBatch(heads + 1, [9000, 5, 7777, 64], [1, 2, 1, 3], heads, rank, 128))


def test_every_key_counts_once():
    """With q = 0 every visible key has the same probability: L = log n, and O is the
    mean of whole numbers, exact but for the division (2^-23), the rounding of
    P's weight 1 (none) and of O (2^-8).  One key too many or too few shows in L."""
    r = np.random.default_rng(3)
    for heads, rank, page, lens, news in [
            (16, 512, 64, [1, 2, 63, 64, 65, 1000, 4095, 129, 20000], [1] * 9), (128, 512, 32, [77, 700, 1500], [1, 4, 2]),
            (7, 256, 128, [3000, 130, 128, 127], [40, 130, 1, 9]), (64, 256, 64, [100] * 200, [1] * 200)]:
        b = LatentBatch(int(r.integers(1 << 30)), lens, news, heads, rank, page, pad_rows=1, whole=True)
        b.q[:] = 0.0
        for causal, x in ((c, x) for c in (True, False) for x in b.tables()):
            o, l = run(x, causal)
            for s, (t, n) in enumerate(zip(lens, news)):
                v = C.tokens(b.data, b.table[s], t)[:, :rank]
                for i in range(n):
                    see = t - n + i + 1 if causal else t
                    row = int(b.q_start[s]) + i
                    assert (np.abs(l[row] - np.log(see)) <= 2.0 ** -22 * max(1.0, np.log(see))).all()
                    mean = v[:see].sum(axis=0) / see
                    assert (np.abs(o[row] - mean) <= (2.0 ** -8 + 2.0 ** -21) * np.abs(mean)).all()


@pytest.mark.parametrize("heads", [16, 128])
def test_one_key_takes_all(heads):
    """A score far above the others, at each place of the tiles in turn: O is that key's
    latent, to the rounding, whichever CTA and tile it lies in."""
    lens = [64 * 37 + 5]
    b = LatentBatch(9, lens, [1], heads, 512, 64)
    b.data = np.nan_to_num(b.data, nan=3.0)
    for at in (0, 1, 63, 64, 700, 64 * 36 + 63, 64 * 37, 64 * 37 + 4):
        data = b.data.copy()
        data[..., -1] = 0.0
        data[b.table[0, at // 64], at % 64, -1] = 64.0
        b2 = LatentBatch(9, lens, [1], heads, 512, 64)
        b2.data, b2.q = data, b.q * 0.0
        b2.q[..., -1] = 64.0
        for x in b2.tables():
            o, l = run(x, scale=0.1)
            assert np.array_equal(o[0], np.broadcast_to(data[b.table[0, at // 64], at % 64, :512], o[0].shape))
            assert (np.abs(l - 409.6) <= 409.6 * 2.0 ** -21).all()


@pytest.mark.parametrize("scale_q", [20.0, 0.01])
@pytest.mark.parametrize("heads", [16, 128])
def test_large_and_small_scores(scale_q, heads):
    """Scores of several hundred whose running maximum keeps moving, and tiny ones."""
    check(LatentBatch(21, [2000, 100], [1, 3], heads, 512, 64, scale_q=scale_q))


@pytest.mark.parametrize("heads,rank", [(20, 256), (128, 512)])
def test_rising_scores_move_the_reference_in_every_tile(heads, rank):
    b = LatentBatch(22, [64 * 12], [1], heads, rank, 64)
    for i in range(64 * 12):
        b.data[b.table[0, i // 64], i % 64, -1] = i // 4      # whole numbers below 256: bf16 has them
    b.q[..., -1] = 8.0
    check(b, scale=0.1)


@pytest.mark.parametrize("n,news", [(33, 1), (300, 2), (1100, 1), (4096, 1)])
def test_many_sequences(n, news):
    r = np.random.default_rng(n)
    lens = [int(x) for x in r.integers(news, 90, n)]
    b = LatentBatch(n, lens, [news if i % 7 else 0 for i in range(n)], 3, 256, 32, pad_rows=3)
    check(b)


def test_rows_that_see_nothing():
    """Empty caches, rows before the first position, empty sequences in between."""
    for heads in (3, 80):
        o, l, want = check(LatentBatch(31, [0, 5, 3, 130, 0], [3, 9, 1, 1, 0], heads, 512, 32, pad_rows=2))
        assert np.isneginf(want[1][:3]).all() and np.isneginf(want[1][3:7]).all()
        check(LatentBatch(32, [0, 5], [3, 9], heads, 256, 64), causal=False)


@pytest.mark.parametrize("heads,page", [(16, 64), (128, 32), (128, 128)])
def test_gaps_between_pages_and_wide_tables(heads, page):
    b = LatentBatch(33, [200, 513], [1, 1], heads, 512, page)
    check(b, gap=64)
    b.table = np.concatenate([b.table, np.full((2, 3000), -7, np.int32)], axis=1)
    check(b)


@pytest.mark.parametrize("heads", [3, 16, 64, 128])
def test_no_rows_at_all(heads):
    """Only padding: nothing is written, in any layout."""
    b = LatentBatch(45, [70, 300], [0, 0], heads, 512, 64, pad_rows=3)
    for x in b.tables():
        o, l = run(x)
        assert (o == 7.0).all() and (l == 7.0).all()


@pytest.mark.parametrize("heads,pages,page", [(16, 3, 32), (64, 5, 64), (128, 608, 128)])
def test_tables_that_are_full(heads, pages, page):
    """Lengths that fill the table to its last slot (128 heads: on pairs)."""
    b = LatentBatch(46, [pages * page], [1], heads, 512, page)
    b.table, b.max_pages = np.ascontiguousarray(b.table[:, :pages]), pages
    o, l = run(b)
    check_latent(o, l, C.attend(b.q, b.data, 512, b.table, b.q_start, b.kv_len, True, 0.07), 576)


def test_many_sequences_of_many_rows():
    """More sequences than a pair has threads, and most heads."""
    r = np.random.default_rng(47)
    lens = [int(x) for x in r.integers(1, 40, 700)]
    check(LatentBatch(47, lens, [1 if i % 7 else 0 for i in range(700)], 80, 512, 32, pad_rows=3))
    check(LatentBatch(48, [90, 5], [1, 2], 1024, 512, 64))


def test_pages_that_do_not_exist():
    """Tokens of missing pages count as absent and are reported; also where a row
    then sees nothing."""
    for page, heads in ((32, 16), (64, 16), (128, 16), (32, 128), (128, 128)):
        b = LatentBatch(34, [700, 90, 300, 20], [1, 1, 2, 1], heads, 512, page)
        b.table[0, 1], b.table[2, 0], b.table[3, 0] = b.pages, -3, 1 << 30
        want = C.attend(b.q, b.data, b.rank, b.table, b.q_start, b.kv_len, True, 0.07)
        for x in b.tables():
            c, *where = x.device()
            o, l = F.fattn_latent_fwd(b.rows(b.q), c, *where, scale=0.07)
            assert F.fattn_check_status() == _lib.FATTN_ERR_BAD_INDEX
            check_latent(*arrays(o, l), want, b.rank + ROPE)
        assert np.isneginf(want[1][-1]).all()
    ok()


@pytest.mark.parametrize("what", ["longer than its table", "negative length", "q_start past the rows", "q_start back"])
@pytest.mark.parametrize("rank", [256, 512])
def test_senseless_sequences(what, rank):
    *_, b = LatentBatch(35, [60, 90, 40], [5, 20, 3], 20, rank, 32).tables()
    c, table, qs, kl = b.device()
    want = F.fattn_latent_fwd(b.rows(b.q), c, table, qs, kl, scale=0.07)
    ok()
    if what == "longer than its table":
        kl[1] = b.max_pages * 32 + 1
    elif what == "negative length":
        kl[1] = -1
    elif what == "q_start past the rows":
        qs[3] = b.T + 1
    else:
        qs[1] = 26
    o, l = F.fattn_latent_fwd(b.rows(b.q), c, table, qs, kl, scale=0.07)
    assert F.fattn_check_status() == _lib.FATTN_ERR_BAD_INDEX
    # the sequences that make sense are served (row 25 belongs to two where q_start goes back)
    good = slice(26, 28) if what == "q_start back" else slice(0, 5)
    assert torch.equal(o[good], want[0][good]) and torch.equal(l[good], want[1][good])
    ok()


@pytest.mark.parametrize("heads,news,rank", [(3, 1, 256), (3, 3, 256), (40, 2, 256), (128, 1, 256), (128, 1, 512), (128, 3, 512)])
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_infinite_queries(heads, news, rank, bad):
    """A query with an infinity has infinite scores and so a NaN row, also where all of
    them are -inf; it is no row that sees nothing.  Other rows and heads stay."""
    *_, b = LatentBatch(36, [150, 70], [news, news], heads, rank, 32).tables()
    b.data[..., 9] = np.abs(b.data[..., 9]) + 0.5       # one sign: all scores are inf, or all -inf
    c, *where = b.device()
    o0, l0 = F.fattn_latent_fwd(b.rows(b.q), c, *where, scale=0.07)
    row = news // 2
    b.q[row, 1, 9] = bad
    for causal in (True, False):
        o, l = F.fattn_latent_fwd(b.rows(b.q), c, *where, scale=0.07, causal=causal)
        assert bool(torch.isnan(o[row, 1]).all()) and bool(torch.isnan(l[row, 1]))
        assert int(torch.isnan(l).sum()) == 1
        if causal:
            keep = torch.ones((b.T, heads), dtype=torch.bool, device="cuda")
            keep[row, 1] = False
            assert torch.equal(o[keep], o0[keep]) and torch.equal(l[keep], l0[keep])
    ok()


def test_infinite_query_over_many_ctas():
    b = LatentBatch(37, [9000], [1], 16, 512, 64)
    b.data[..., 9] = np.abs(b.data[..., 9]) + 0.5
    b.q[0, 3, 9] = -np.inf
    o, l = run(b)
    assert np.isnan(l[0, 3]) and np.isnan(o[0, 3]).all() and np.isfinite(np.delete(l[0], 3)).all()


@pytest.mark.parametrize("kernel", [0, 1])
def test_same_bits_every_time_and_in_any_company(kernel):
    b = list(LatentBatch(38, [5000, 130, 777], [1, 2, 1], 128, 512, 64).tables())[kernel]
    c, *where = b.device()
    q = b.rows(b.q)
    first = F.fattn_latent_fwd(q, c, *where, scale=0.07)
    ws = torch.full((F.fattn_latent_fwd_workspace_bytes(4, 3, 128, 512),), 0xFF, dtype=torch.uint8, device="cuda")
    for i in range(6):
        got = F.fattn_latent_fwd(q, c, *where, scale=0.07, workspace=ws if i & 1 else None)
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
    ok()


def test_offsets_past_32_bits():
    """Pages whose bytes and elements lie past 2^31 and 2^32."""
    pages, page = 62000, 64
    data = torch.empty((pages, page, 576), dtype=torch.bfloat16, device="cuda")
    b = LatentBatch(39, [300, 70], [1, 2], 16, 512, page, spare=0)
    ids = np.array([61999, 3, 60000, 30000, 58255, 61000, 59000])
    where = torch.from_numpy(ids[:b.pages]).cuda()
    data[where] = torch.from_numpy(b.data).to(torch.bfloat16).cuda()
    table = np.where(b.table < b.pages, ids[np.minimum(b.table, b.pages - 1)], b.table).astype(np.int32)
    rest = [torch.from_numpy(x).cuda() for x in (table, b.q_start, b.kv_len)]
    o, l = F.fattn_latent_fwd(b.rows(b.q), F.LatentCache(data, 512), *rest, scale=0.07)
    ok()
    want = C.attend(b.q, b.data, 512, b.table, b.q_start, b.kv_len, True, 0.07)
    check_latent(*arrays(o, l), want, 576)
    lat, key = b.rows(b.latent), b.rows(b.k_rope)
    F.fattn_latent_append(lat, key, F.LatentCache(data, 512), *rest)
    ok()
    assert torch.equal(data[int(table[0, 4]), 299 % 64, :512], lat[0])


def test_offsets_past_32_bits_on_pairs():
    pages, page = 62000, 64
    data = torch.empty((pages, page, 576), dtype=torch.bfloat16, device="cuda")
    *_, b = LatentBatch(44, [300, 70], [1, 2], 128, 512, page, spare=0).tables()
    ids = np.array([61999, 3, 60000, 30000, 58255, 61000, 59000])
    data[torch.from_numpy(ids[:b.pages]).cuda()] = torch.from_numpy(b.data).to(torch.bfloat16).cuda()
    table = np.where(b.table < b.pages, ids[np.minimum(b.table, b.pages - 1)], b.table).astype(np.int32)
    rest = [torch.from_numpy(x).cuda() for x in (table, b.q_start, b.kv_len)]
    o, l = F.fattn_latent_fwd(b.rows(b.q), F.LatentCache(data, 512), *rest, scale=0.07)
    ok()
    check_latent(*arrays(o, l), C.attend(b.q, b.data, 512, b.table, b.q_start, b.kv_len, True, 0.07), 576)


def test_random_batches():
    r = np.random.default_rng(40)
    for i in range(25):
        n = int(r.integers(1, 9))
        lens = [int(x) for x in r.integers(1, 900, n)]
        news = [int(min(t, r.choice([0, 1, 1, 2, 5, 40]))) for t in lens]
        if not sum(news):
            news[0] = 1
        heads = int(r.choice([1, 2, 7, 16, 31, 48, 65, 128]))
        b = LatentBatch(1000 + i, lens, news, heads, int(r.choice([256, 512])), int(r.choice([32, 64, 128])), pad_rows=int(i % 3))
        check(b, causal=bool(i % 4))


# ------------------------------------------------------------------ append

def run_append(b, rope=True, interleaved=False, with_q=True, gap=0, fused=True):
    c, *where = b.device(gap)
    t = F.fattn_rope_table(max(b.lens) + 3, 64) if rope else None
    lat, key = b.rows(b.latent), b.rows(b.k_rope)
    if fused:
        one = torch.cat([lat, key], dim=1)
        lat, key = one[:, :b.rank], one[:, b.rank:]
    qr = torch.cat([torch.zeros((b.T, b.heads, 24), device="cuda", dtype=torch.bfloat16), b.rows(b.q_rope)], dim=2)[:, :, 24:]
    q = b.rows(b.q) if with_q else None
    F.fattn_latent_append(lat, key, c, *where, rope=t, q_rope=qr if with_q else None, q=q, interleaved=interleaved)
    return c, q, None if t is None else t.cpu().numpy()


def check_append(b, **kw):
    c, q, t = run_append(b, **kw)
    ok()
    data, want_q = b.data.copy(), b.q.copy()
    n = int(b.q_start[-1])
    C.append(data, b.latent, b.k_rope, b.table, b.q_start, b.kv_len, t, kw.get("interleaved", False), b.q_rope, want_q)
    assert np.array_equal(c.data.float().cpu().numpy(), data, equal_nan=True)
    if q is not None:
        assert np.array_equal(q.float().cpu().numpy(), want_q)     # other columns and padding rows as they were


@pytest.mark.parametrize("rank,page", [(256, 32), (256, 128), (512, 64), (512, 128)])
@pytest.mark.parametrize("lens,news,heads", [
    ([1], [1], 1), ([33, 128, 1, 65], [1, 1, 1, 1], 16), ([300, 129, 64], [300, 2, 64], 5), ([257, 31, 500], [130, 0, 77], 128)])
def test_append(rank, page, lens, news, heads):
    b = LatentBatch(sum(lens) + rank + page, lens, news, heads, rank, page, pad_rows=3)
    check_append(b, interleaved=bool(len(lens) & 1))


@pytest.mark.parametrize("kw", [dict(rope=False), dict(with_q=False), dict(gap=64), dict(interleaved=True), dict(fused=False)])
def test_append_variants(kw):
    check_append(LatentBatch(50, [100, 40, 0, 9], [50, 1, 0, 9], 3, 256, 32, pad_rows=1), **kw)


def test_append_many_sequences_and_in_place():
    r = np.random.default_rng(51)
    lens = [int(x) for x in r.integers(1, 40, 2000)]
    check_append(LatentBatch(51, lens, [int(r.integers(0, t + 1)) for t in lens], 1, 256, 32, pad_rows=2))
    b = LatentBatch(52, [70, 30], [70, 3], 9, 512, 64)
    c, *where = b.device()
    q = b.rows(b.q)
    t = F.fattn_rope_table(80, 64)
    F.fattn_latent_append(b.rows(b.latent), b.rows(b.k_rope), c, *where, rope=t, q_rope=q[:, :, 512:], q=q)
    ok()
    want = b.q.copy()
    C.append(b.data.copy(), b.latent, b.k_rope, b.table, b.q_start, b.kv_len, t.cpu().numpy(), False, b.q[:, :, 512:].copy(), want)
    assert np.array_equal(q.float().cpu().numpy(), want)


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("column", [0, 255, 256, 511, 512, 575])
def test_tokens_that_are_not_finite(bad, column):
    """Such a token makes the rows that attend to it NaN, and no others."""
    *_, b = LatentBatch(53, [90, 70], [40, 3], 4, 512, 32).tables()
    if column < 512:
        b.latent[20, column] = bad
    else:
        b.k_rope[20, column - 512] = bad
    check_append(b)
    c, q, _ = run_append(b)
    _, *where = b.device()
    o, l = F.fattn_latent_fwd(q, c, *where, scale=0.07)
    ok()
    nan = torch.zeros(b.T, dtype=torch.bool, device="cuda")
    nan[20:40] = True
    assert torch.equal(torch.isnan(l).all(dim=1), nan) and torch.equal(torch.isnan(l).any(dim=1), nan)
    assert torch.equal(torch.isnan(o).all(dim=2).all(dim=1), nan) and torch.equal(torch.isnan(o).any(dim=2).any(dim=1), nan)


@pytest.mark.parametrize("what", ["longer than its table", "negative length", "more new than cached", "past the rotation's table",
                                  "a page outside", "q_start back"])
def test_append_leaves_senseless_sequences_alone(what):
    b = LatentBatch(54, [60, 90, 40], [5, 40, 3], 2, 256, 32)
    c, table, qs, kl = b.device()
    t = F.fattn_rope_table(70 if what == "past the rotation's table" else 400, 64)
    q = b.rows(b.q)
    if what == "longer than its table":
        kl[1] = b.max_pages * 32 + 1
    elif what == "negative length":
        kl[1] = -1
    elif what == "more new than cached":
        kl[1] = 39
    elif what == "a page outside":
        table[1, 1:3] = b.pages
    elif what == "q_start back":
        qs[2] = 3
    before = c.data.clone()
    F.fattn_latent_append(b.rows(b.latent), b.rows(b.k_rope), c, table, qs, kl, rope=t, q_rope=b.rows(b.q_rope), q=q)
    assert F.fattn_check_status() == _lib.FATTN_ERR_BAD_INDEX
    pages = torch.from_numpy(b.table[1, :3]).cuda().long()
    same = torch.equal(c.data[pages].view(torch.int16), before[pages].view(torch.int16))
    if what != "a page outside":
        assert same
        if what != "q_start back":
            assert torch.equal(q[5:45], b.rows(b.q)[5:45])
    else:
        assert torch.equal(c.data[pages[1:]].view(torch.int16), before[pages[1:]].view(torch.int16))
    want_q, data = b.q.copy(), b.data.copy()
    C.append(data, b.latent[:5], b.k_rope[:5], b.table[:1], b.q_start[:2], b.kv_len[:1], t.cpu().numpy(), False, b.q_rope[:5], want_q)
    assert np.array_equal(c.data[b.table[0, 1]].float().cpu().numpy(), data[b.table[0, 1]], equal_nan=True)
    ok()
