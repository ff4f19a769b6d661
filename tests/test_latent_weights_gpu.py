"""The latent attention's weights add up to one: where all values are equal, O is that value,
however far the probabilities' rounding carries them, and whichever kernel, tile and
share they come from."""

import numpy as np
import pytest
import torch

import exact_attention_fattn_gb300 as F

pytestmark = pytest.mark.gpu

V = 255 / 128      # the last number below 2: half a step of bf16 is 2^-9 of it, the least there is


def batch(n, length, heads, rank, room, page=64):
    """n sequences of `length` keys with the same value: key 0 scores 0 and the others far less, but
    for one in the last tile that scores above it, by less than what moves a reference."""
    per = -(-length // page)
    cache = F.fattn_latent_alloc(n * per, rank, page)
    cache.data[..., :rank] = V
    cache.data[..., -1] = -32.0
    table = torch.full((n, max(per, room // page)), -1, dtype=torch.int32, device="cuda")
    table[:, :per] = torch.arange(n * per, dtype=torch.int32, device="cuda").view(n, per)
    cache.data[table[:, 0].long(), 0, -1] = 0.0
    cache.data[table[:, per - 1].long(), (length - 1) % page, -1] = 1.0
    q = torch.zeros((n, heads, rank + 64), dtype=torch.bfloat16, device="cuda")
    q[..., -1] = 0.5 + torch.arange(n * heads, device="cuda").view(n, heads).remainder(64) / 128.0
    where = [torch.arange(n + 1, dtype=torch.int32, device="cuda"), torch.full((n,), length, dtype=torch.int32, device="cuda")]
    return q, cache, table, where


@pytest.mark.parametrize("rank,heads,room", [(256, 16, 0), (512, 16, 0), (512, 32, 0), (256, 64, 0), (512, 64, 0), (512, 128, 0),
                                             (512, 128, 120000)])
@pytest.mark.parametrize("n,length", [(300, 385), (300, 200), (1, 3000), (40, 2000)])
def test_equal_values(n, length, heads, rank, room):
    q, cache, table, where = batch(n, length, heads, rank, room)
    scale = 5.5                            # 2^7.93 at most above key 0
    o, lse = F.fattn_latent_fwd(q, cache, table, *where, scale=scale)
    assert F.fattn_check_status() == 0
    # Products of bf16 numbers are exact in fp32; their sums, the rounded probabilities' and the
    # division are off by less than (length + 8) 2^-23, under 2^-9 of V: the rounding to bf16
    # gives V.
    assert (length + 8) * 2.0 ** -23 < 2.0 ** -10
    assert bool((o == V).all()), float((o.float() - V).abs().max())
    s = q[..., -1].double().cpu().numpy() * scale
    # The far keys have e^-88 at most.  A score has one product, so that L's error is that of the
    # scaling (2^-23 of 5.5), the exponential (2^-22), the sum and the logarithm (2^-22 of L), L >= 2.8.
    want = np.log1p(np.exp(s) + (length - 2) * np.exp(-32.0 * s))
    assert (np.abs(lse.double().cpu().numpy() - want) <= 2.0 ** -19 * want).all()
