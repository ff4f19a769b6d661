"""A wait budget that is far too short: the latent cache's attention gives up and says so, a call
that says it is fine is right, and the next call with the usual budget is right."""

import pytest
import torch

import exact_attention_fattn_gb300 as F
import test_pages_gpu as P
from exact_attention_fattn_gb300 import _lib
from latent_util import LatentBatch

pytestmark = pytest.mark.gpu


@pytest.fixture
def budget():
    try:
        yield F.fattn_set_wait_budget
    finally:
        F.fattn_set_wait_budget(0)


@pytest.mark.parametrize("page", [32, 64])
@pytest.mark.parametrize("news,heads", [(1, 16), (1, 40), (1, 128), (60, 20)])
def test_attention_that_says_it_is_fine_is_right(news, heads, page, budget):
    """Few tiles, so that waits may be over at their first look, whatever the budget."""
    *_, b = LatentBatch(80, [3000, 700], [news, news], heads, 512, page).tables()
    dev, q = b.device(), b.rows(b.q)
    want = F.fattn_latent_fwd(q, *dev, scale=0.07)
    assert F.fattn_check_status() == 0
    for cycles in (1, 200, 1500, 4000, 20000, 1 << 20):
        budget(cycles)
        for _ in range(3):
            got = F.fattn_latent_fwd(q, *dev, scale=0.07)
            rc = F.fattn_check_status()
            assert rc in (_lib.FATTN_OK, _lib.FATTN_ERR_TIMEOUT)
            if rc == _lib.FATTN_OK:
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    budget(0)
    got = F.fattn_latent_fwd(q, *dev, scale=0.07)
    assert F.fattn_check_status() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("page", [32, 64])
@pytest.mark.parametrize("heads", [16, 64, 128])
def test_attention_that_gives_up_says_so(heads, page, budget):
    """340 MB of cached tokens, more than L2 holds: every CTA is ahead of its copies at most of its
    tiles, where the products' issue polls, and so gives up after one cycle."""
    n, length = 48, 6000
    per = -(-length // page)
    cache = F.LatentCache(torch.randn((n * per, page, 576), device="cuda").to(torch.bfloat16), 512)
    table = torch.arange(n * per, dtype=torch.int32, device="cuda").view(n, per)
    where = [torch.arange(n + 1, dtype=torch.int32, device="cuda"), torch.full((n,), length, dtype=torch.int32, device="cuda")]
    q = torch.randn((n, heads, 576), device="cuda").to(torch.bfloat16)
    want = F.fattn_latent_fwd(q, cache, table, *where, scale=0.07)
    assert F.fattn_check_status() == 0
    budget(1)
    for _ in range(3):
        F.fattn_latent_fwd(q, cache, table, *where, scale=0.07)
        assert F.fattn_check_status() == _lib.FATTN_ERR_TIMEOUT
    budget(0)
    got = F.fattn_latent_fwd(q, cache, table, *where, scale=0.07)
    assert F.fattn_check_status() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_copies_that_say_they_are_fine_are_right(budget):
    """A copy's wait suspends its thread until the copy lands or a limit of the hardware's, so it may
    outlast any budget; but then the pages are right."""
    for i in range(6):
        p = P.Pool("latent", 400, 20, 12, 128, seed=i)
        p.extend([100 + 50 * j for j in range(20)])
        p.free(list(range(0, 20, 2)))
        budget(1)
        p.compact()
        rc = F.fattn_check_status()
        budget(0)
        assert rc in (_lib.FATTN_OK, _lib.FATTN_ERR_TIMEOUT)
        if rc == _lib.FATTN_OK:
            p.same()
