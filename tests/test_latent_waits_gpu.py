"""Batches on which the roles of the latent attention's kernels have to wait for one
another at every tile: references that move in each of them, sequences whose last
tiles have one page or two."""

import numpy as np
import pytest
import torch

import exact_attention_fattn_gb300 as F
import oracle
from latent_util import ROPE, LatentBatch, check_latent

pytestmark = pytest.mark.gpu


def attend(b, scale, causal=True):
    c, *where = b.device()
    return F.fattn_latent_fwd(b.rows(b.q), c, *where, scale=scale, causal=causal)


def check(b, scale=0.07):
    want = oracle.latent.attend(b.q, b.data, b.rank, b.table, b.q_start, b.kv_len, True, scale)
    for x in b.tables():
        o, lse = attend(x, scale)
        assert F.fattn_check_status() == 0
        check_latent(o.double().cpu().numpy(), lse.double().cpu().numpy(), want, b.rank + ROPE)


@pytest.mark.parametrize("step", [1, 4, 97])
@pytest.mark.parametrize("page", [64, 128])
def test_references_that_move_in_every_tile(page, step):
    """Scores that rise with the key, for some rows by more than 2^8 a tile and for others
    not at all, so that O is rescaled in each tile while other warps' rows stay: within the
    bound, and the same bits every time."""
    lens, news = [64 * 30 + 7, 64 * 21], [1, 2]
    b = LatentBatch(500 + step, lens, news, 128, 512, page)
    for s, t in enumerate(lens):
        for i in range(t):
            b.data[b.table[s, i // page], i % page, -1] = float(i // 8)       # whole numbers below 256
    b.q[..., -1] = (np.arange(b.q.shape[1]) * step % 8).astype(np.float32)
    check(b, scale=0.4)
    *_, wide = b.tables()
    c, *where = wide.device()
    q = wide.rows(wide.q)
    first = F.fattn_latent_fwd(q, c, *where, scale=0.4)
    for _ in range(40):
        got = F.fattn_latent_fwd(q, c, *where, scale=0.4)
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
    assert F.fattn_check_status() == 0


@pytest.mark.parametrize("rank,heads", [(256, 16), (512, 16), (256, 40), (512, 64), (512, 20)])
def test_tiles_of_one_page_and_of_two_in_turn(rank, heads):
    """Pages of 32 tokens: many sequences of up to 32, which have one, among some of up to 64 and
    of a few tiles; the warp of the second pages must not miss its turn."""
    r = np.random.default_rng(rank + heads)
    short = [int(x) for x in r.integers(1, 33, 900)]
    lens = [int(r.integers(33, 65)) if i % 9 == 8 else (int(r.integers(65, 400)) if i % 50 == 20 else t) for i, t in enumerate(short)]
    b = LatentBatch(510 + heads, lens, [1] * len(lens), heads, rank, 32)
    check(b)
    c, *where = b.device()
    q = b.rows(b.q)
    first = F.fattn_latent_fwd(q, c, *where, scale=0.07)
    for _ in range(20):
        got = F.fattn_latent_fwd(q, c, *where, scale=0.07)
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
    assert F.fattn_check_status() == 0
