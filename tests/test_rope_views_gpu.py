"""Rotations of views whose strides say little: dimensions of one."""

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
