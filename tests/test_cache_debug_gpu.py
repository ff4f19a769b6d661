"""The paged cache on the checked debug variant of the library: every kernel
range-checks the indices it computes (workspace slots, rows of the outputs,
shared-memory and page offsets; a failed check would be FATTN_ERR_DEBUG_CHECK),
and the many-rows kernel's K ring has two stages.  The cases are those of
test_cache_gpu.py where indices go to their edges; results must still match
the oracle, and no check may fire."""

import numpy as np
import pytest
import torch

import test_cache_gpu as T
from cache_util import Batch
from exact_attention_fattn_gb300 import _lib, build
from exact_attention_fattn_gb300 import cache as K

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def debug_lib():
    lib = _lib.load(build.build(debug=True))
    saved = _lib._lib
    _lib._lib = lib
    K.fattn_cache_fwd_workspace_bytes.cache_clear()
    try:
        yield lib
    finally:
        _lib._lib = saved


@pytest.mark.parametrize("d,page", [(64, 32), (64, 64), (128, 64), (128, 128)])
def test_append(d, page):
    T.check_append(Batch(400 + page, [300, 129, 64, 1], [300, 2, 64, 1], 2, 3, d, page, pad_rows=3, filled=False),
                   rope_dim=d)
    T.check_append(Batch(401, [257, 31, 500], [130, 0, 77], 2, 9, d, page, filled=False), rope_dim=48,
                   interleaved=True, page_gap=48)


@pytest.mark.parametrize("d,page", [(64, 32), (64, 128), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_attend(d, page, causal):
    # single tokens; rows around the tiles' ends; few rows on many keys, shared by many CTAs
    T.check(Batch(410, [1, 31, 32, 33, 257, 600, 1029], [1] * 7, 2, 7, d, page, pad_rows=2), causal)
    T.check(Batch(411, [65, 256, 134, 257, 1, 500, 300, 128, 390], [65, 128, 129, 255, 1, 257, 300, 127, 66], 2, 1, d,
                  page), causal)
    T.check(Batch(412, [9000, 777], [20, 9], 1, 8, d, page), causal)
    T.check(Batch(413, [12000, 5, 3000], [1, 1, 1], 2, 2, d, page), causal)
    T.check(Batch(414, [0, 5, 3, 130], [3, 9, 200, 1], 2, 2, d, page, pad_rows=2), causal)


@pytest.mark.parametrize("news,g", [(1, 2), (5, 16)])
def test_most_sequences(news, g):
    r = np.random.default_rng(143)
    lens = [int(x) for x in r.integers(news, 40, 4096)]
    b = Batch(143, lens, [news if i % 7 else 0 for i in range(4096)], 1, g, 128, 32, pad_rows=3)
    T.check(b)
    sel = np.zeros((b.T, 1, 2), np.int32)
    sel[:, :, 1] = -1
    T.check(b, selected=sel)


@pytest.mark.parametrize("news", [[1, 1], [30, 2]])
def test_largest_group_and_most_heads(news):
    T.check(Batch(420, [300, 129], news, 1, 128, 128, 64, pad_rows=1))
    T.check(Batch(421, [70, 33], news, 1024, 1, 64, 32))


@pytest.mark.parametrize("lens,news,hkv,k", [
    ([2300 * 32], [2], 1, 20), ([2300 * 32 - 5, 70], [70, 2], 1, 20), ([500 * 32 - 3, 9000], [30, 150], 2, 20),
    ([10400 * 32 - 31], [80], 2, 40), ([32 * 5, 1, 0], [2, 1, 1], 2, 8)])
def test_select_and_attend_to_the_selection(lens, news, hkv, k):
    b = Batch(430, lens, news, hkv, 2, 64, 32, pad_rows=1)
    want = T.C.select(b.q, b.cache, b.table, b.q_start, b.kv_len, k, 1, 2)
    got = T.run_select(b, k, 1, 2)
    assert np.array_equal(got, want)
    if max(lens) < 100000:
        T.check(b, selected=np.where(got == -2, -1, got).astype(np.int32))


def test_captured_step():
    b = Batch(440, [900, 300], [60, 60], 1, 4, 128, 64)
    c, *where = b.device()
    q = b.rows(b.q)
    want = K.fattn_cache_fwd(q, c, *where)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = K.fattn_cache_fwd(q, c, *where)
    g.replay()
    T.status_ok()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
