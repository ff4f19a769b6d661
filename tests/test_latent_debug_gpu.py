"""The latent cache, the pages and the rotations on the checked debug variant of
the library: every kernel range-checks the indices it computes, and the ring of
cached tokens has its least depth of two tiles.  The cases are those of the other
files where indices go to their edges; no check may fire."""

import numpy as np
import pytest
import torch

import exact_attention_fattn_gb300 as F
import test_latent_gpu as T
import test_pages_gpu as P
from exact_attention_fattn_gb300 import _lib, build
from latent_util import LatentBatch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def debug_lib():
    lib = _lib.load(build.build(debug=True))
    saved = _lib._lib
    _lib._lib = lib
    try:
        yield lib
    finally:
        _lib._lib = saved


@pytest.mark.parametrize("rank,page", [(256, 32), (256, 128), (512, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_attend(rank, page, causal):
    T.check(LatentBatch(400, [1, 31, 32, 33, 257, 600, 1029], [1] * 7, 7, rank, page, pad_rows=2), causal)
    T.check(LatentBatch(401, [65, 256, 134, 257, 1, 500], [65, 128, 129, 255, 1, 257], 1, rank, page), causal)
    T.check(LatentBatch(402, [9000, 777], [1, 3], 128, rank, page), causal)
    T.check(LatentBatch(403, [12000, 5, 3000], [1, 1, 1], 20, rank, page), causal)
    T.check(LatentBatch(404, [0, 5, 3, 130], [3, 9, 200, 1], 33, rank, page, pad_rows=2), causal)
    T.check(LatentBatch(405, [400], [400], 64, rank, page), causal)


def test_most_sequences():
    r = np.random.default_rng(143)
    lens = [int(x) for x in r.integers(1, 40, 4096)]
    T.check(LatentBatch(143, lens, [1 if i % 7 else 0 for i in range(4096)], 16, 256, 32, pad_rows=3))


@pytest.mark.parametrize("rank,page", [(256, 32), (512, 64), (512, 128)])
def test_append(rank, page):
    T.check_append(LatentBatch(410, [300, 129, 64, 1], [300, 2, 64, 1], 3, rank, page, pad_rows=3))
    T.check_append(LatentBatch(411, [257, 31, 500], [130, 0, 77], 9, rank, page), interleaved=True, gap=64)


@pytest.mark.parametrize("kw", P.KINDS)
def test_pages(kw):
    P.test_a_life(kw, 32)


def test_many_pages():
    P.test_many_sequences_and_pages()
    P.test_a_pool_of_a_million_pages()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope(interleaved):
    t = F.fattn_rope_table(300, 48)
    for shape in ((1, 1, 1, 64), (2, 9, 257, 128), (3, 5, 33, 48)):
        x = torch.randn(shape, device="cuda").to(torch.bfloat16)
        y = F.fattn_rope(x, t, interleaved=interleaved)
        F.fattn_rope_bwd(y, t, interleaved=interleaved, out=y)
    T.ok()


def test_captured_step():
    *_, b = LatentBatch(440, [900, 300], [2, 1], 100, 512, 64).tables()
    c, *where = b.device()
    q = b.rows(b.q)
    want = F.fattn_latent_fwd(q, c, *where, scale=0.1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = F.fattn_latent_fwd(q, c, *where, scale=0.1)
    g.replay()
    T.ok()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
