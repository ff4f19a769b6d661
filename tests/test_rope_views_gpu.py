"""Rotations of views whose strides say little: dimensions of one, and tensors past 32
bits of elements, first and last row against the oracle."""

import numpy as np
import pytest
import torch

import exact_attention_fattn_gb300 as F
import oracle
from cache_util import to_bf16

pytestmark = pytest.mark.gpu


def turned(x, table, at, interleaved=False, back=False):
    """Rows [..., d] of positions `at`, bit for bit."""
    return torch.from_numpy(to_bf16(oracle.rope.rotate_fp32(x.float().cpu().numpy(), table.cpu().numpy()[at], interleaved, back)))


@pytest.mark.parametrize("view", [
    lambda x: x.reshape(3, 4, 64, 1).mT,                          # [3, 4, 1, 64], rows 1 element apart
    lambda x: torch.as_strided(x, (1, 4, 3, 64), (7, 64, 256, 1)),
    lambda x: torch.as_strided(x, (3, 1, 4, 64), (256, 3, 64, 1)),
    lambda x: torch.as_strided(x, (1, 1, 1, 64), (1, 5, 9, 1)),
    lambda x: torch.as_strided(x, (1, 4, 64), (1, 64, 1)),        # rows [T, H, d]
    lambda x: torch.as_strided(x, (4, 1, 64), (64, 1, 1))])
@pytest.mark.parametrize("call", [F.fattn_rope, F.fattn_rope_bwd])
def test_dimensions_of_one_with_any_stride(view, call):
    torch.manual_seed(1)
    x = view(torch.randn(3 * 4 * 64, device="cuda").to(torch.bfloat16))
    t = F.fattn_rope_table(9, 64)
    n = x.shape[-2] if x.dim() == 4 else x.shape[0]
    at = np.arange(n) if x.dim() == 4 else np.arange(n)[:, None]
    want = turned(x, t, at, back=call is F.fattn_rope_bwd)
    assert torch.equal(call(x, t).float().cpu(), want)
    y = torch.empty_strided(x.shape, x.stride(), dtype=torch.bfloat16, device="cuda") if x.shape[0] == 3 else x.clone()
    assert torch.equal(call(x, t, out=y).float().cpu(), want)
    assert torch.equal(call(x, t, out=x).float().cpu(), want)     # in place
    assert F.fattn_check_status() == 0


@pytest.mark.parametrize("interleaved", [False, True])
def test_rows_past_32_bits_of_elements(interleaved):
    """The first rows, the last ones and those around 2^31 and 2^32 elements are the oracle's of what
    was there before; none of them stays as it was."""
    B, H, N, d = 33, 32, 32768, 128
    x = torch.empty((B, H, N, d), dtype=torch.bfloat16, device="cuda")
    assert x.numel() > 1 << 32
    x.view(-1, 1 << 20).copy_(torch.arange(1 << 20, device="cuda").remainder(251).to(torch.bfloat16))
    t = F.fattn_rope_table(N, d)
    flat = x.view(-1, d)
    rows = sorted({r + k for r in (0, (1 << 31) // d, (1 << 32) // d, B * H * N) for k in (-3, -2, -1, 0, 1, 2)
                   if 0 <= r + k < B * H * N})
    at = torch.tensor(rows, device="cuda")
    flat[at] += torch.randn(len(rows), d, device="cuda").to(torch.bfloat16)
    before = flat[at].clone()
    assert F.fattn_rope(x, t, interleaved=interleaved, out=x) is x
    assert F.fattn_check_status() == 0
    pos = np.array([r % N for r in rows])
    got = flat[at].float().cpu()
    assert torch.equal(got, turned(before, t, pos, interleaved))
    moved = (got != before.float().cpu()).any(dim=1).numpy()
    assert (moved == (pos > 0)).all()                             # position 0 turns by nothing
