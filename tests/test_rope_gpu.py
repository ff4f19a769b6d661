"""Rotary positions on the GPU: bit for bit against the stepwise fp32 oracle and
its one rounding to bf16, over layouts, strides, positions and both directions;
gradients against the formula's and against differences."""

import numpy as np
import pytest
import torch

import exact_attention_fattn_gb300 as F
import oracle
from cache_util import to_bf16
from exact_attention_fattn_gb300 import _lib

pytestmark = pytest.mark.gpu


def ok():
    assert F.fattn_check_status() == 0


def want_of(x, table, at, interleaved, transposed=False):
    """x [B, H, N, d], at [B, N]."""
    return to_bf16(oracle.rope.rotate_fp32(x, table[at][:, None], interleaved, transposed))


def make(seed, shape):
    x = to_bf16(np.random.default_rng(seed).standard_normal(shape))
    return x, torch.from_numpy(x).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("shape,rope_dim", [
    ((1, 1, 1, 64), 64), ((2, 3, 7, 64), 16), ((1, 5, 33, 128), 128), ((3, 1, 257, 128), 64), ((2, 32, 100, 128), 112),
    ((1, 2, 3, 16), 16), ((1, 1, 5, 1024), 1024), ((1, 3, 9, 192), 64), ((2, 9, 1030, 64), 48)])
def test_against_the_formula(shape, rope_dim, interleaved, back):
    x, xd = make(sum(shape) + rope_dim, shape)
    t = F.fattn_rope_table(shape[2] + 5, rope_dim)
    call = F.fattn_rope_bwd if back else F.fattn_rope
    y = call(xd, t, interleaved=interleaved)
    ok()
    at = np.broadcast_to(np.arange(shape[2]), (shape[0], shape[2]))
    assert np.array_equal(y.float().cpu().numpy(), want_of(x, t.cpu().numpy(), at, interleaved, back))
    assert torch.equal(xd.float().cpu(), torch.from_numpy(x))


@pytest.mark.parametrize("interleaved", [False, True])
def test_positions(interleaved):
    r = np.random.default_rng(5)
    x, xd = make(6, (3, 4, 41, 64))
    t = F.fattn_rope_table(130001, 64, factor=8.0, original=4096)
    each = r.integers(0, 130001, (3, 41)).astype(np.int32)
    each[0, 0], each[2, 40] = 0, 130000
    for at in (each, each[1]):
        y = F.fattn_rope(xd, t, positions=torch.from_numpy(at).cuda(), interleaved=interleaved)
        ok()
        assert np.array_equal(y.float().cpu().numpy(), want_of(x, t.cpu().numpy(), np.broadcast_to(at, (3, 41)), interleaved))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 128), (37, 20), (700, 3)])
def test_rows_and_slices(T, H, interleaved):
    """Rows [T, H, d], the last 64 of 192 columns, out of place and in place; what
    lies beside them stays."""
    x, xd = make(T + H, (T, H, 192))
    t = F.fattn_rope_table(T + 9, 64)
    at = torch.randperm(T, generator=torch.Generator().manual_seed(1)).int() + 9
    want = want_of(x[None, :, :, 128:].transpose(0, 2, 1, 3), t.cpu().numpy(), at.numpy()[None], interleaved)[0].transpose(1, 0, 2)
    y = F.fattn_rope(xd[:, :, 128:], t, positions=at.cuda(), interleaved=interleaved)
    assert np.array_equal(y.float().cpu().numpy(), want)
    out = torch.full((T, H, 80), 7.0, dtype=torch.bfloat16, device="cuda")
    F.fattn_rope(xd[:, :, 128:], t, positions=at.cuda(), interleaved=interleaved, out=out[:, :, 16:])
    assert np.array_equal(out[:, :, 16:].float().cpu().numpy(), want) and bool((out[:, :, :16] == 7.0).all())
    z = xd[:, :, 128:]
    assert F.fattn_rope(z, t, positions=at.cuda(), interleaved=interleaved, out=z) is z
    ok()
    assert np.array_equal(xd.float().cpu().numpy(), np.concatenate([x[:, :, :128], want], axis=2))


def test_strides_of_every_kind():
    x, xd = make(9, (2, 6, 50, 64))
    t = F.fattn_rope_table(50, 32)
    want = want_of(x, t.cpu().numpy(), np.broadcast_to(np.arange(50), (2, 50)), False)
    for order in ((0, 1, 2), (0, 2, 1), (1, 0, 2), (1, 2, 0), (2, 0, 1), (2, 1, 0)):
        src = xd.permute(*order, 3).contiguous().permute(*np.argsort(order), 3)
        dst = torch.empty_like(xd.permute(*order[::-1], 3).contiguous()).permute(*np.argsort(order[::-1]), 3)
        F.fattn_rope(src, t, out=dst)
        assert np.array_equal(dst.float().cpu().numpy(), want), order
    one = xd[:, :1].expand(2, 6, 50, 64)          # heads that are one in memory, read only
    y = F.fattn_rope(one, t)
    ok()
    assert np.array_equal(y.float().cpu().numpy(), np.broadcast_to(want[:, :1], want.shape))
    with pytest.raises(_lib.FattnError):
        F.fattn_rope(xd, t, out=one)


def test_positions_outside_the_table_are_left_and_reported():
    x, xd = make(10, (1, 3, 6, 64))
    t = F.fattn_rope_table(8, 64)
    at = np.array([0, 8, 7, -1, 3, 1 << 30], np.int32)
    out = torch.full_like(xd, 7.0)
    F.fattn_rope(xd, t, positions=torch.from_numpy(at).cuda(), out=out)
    assert F.fattn_check_status() == _lib.FATTN_ERR_BAD_INDEX
    got = out.float().cpu().numpy()
    good = [0, 2, 4]
    assert (got[:, :, [1, 3, 5]] == 7.0).all()
    assert np.array_equal(got[:, :, good], want_of(x[:, :, good], t.cpu().numpy(), at[None, good], False))
    F.fattn_rope(xd, F.fattn_rope_table(5, 64))      # a table shorter than the rows
    assert F.fattn_check_status() == _lib.FATTN_ERR_BAD_INDEX
    ok()


@pytest.mark.parametrize("value", [np.inf, np.nan, 3.3e38])
def test_values_at_the_ends(value):
    x, xd = make(11, (1, 2, 9, 64))
    x[0, 1, 4, 3] = value
    xd = torch.from_numpy(x).to(torch.bfloat16).cuda()
    x = xd.float().cpu().numpy()
    t = F.fattn_rope_table(9, 64)
    y = F.fattn_rope(xd, t).float().cpu().numpy()
    want = want_of(x, t.cpu().numpy(), np.arange(9)[None], False)
    assert np.array_equal(y, want, equal_nan=True)
    ok()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kw", [{}, {"factor": 8.0, "original": 4096}])
def test_gradient(interleaved, kw):
    """dx of w . rope(x): the formula's, and differences of the rotation in 64 bits.
    Off by the rounding to bf16 (2^-8 of the value), by fp32's products and sum and
    the table's rounding (4 roundings of 2^-24 of up to 2 max|w| times the magnitude)."""
    r = np.random.default_rng(12)
    B, H, N, d, rd = 1, 2, 7, 64, 32
    w, wd = make(13, (B, H, N, d))
    at = r.integers(0, 100000, (B, N)).astype(np.int32)
    t = F.fattn_rope_table(100000, rd, **kw)
    mag = 0.1 * np.log(8.0) + 1.0 if kw else 1.0
    ang = at[:, None, :, None] * oracle.rope.frequencies(rd, **kw)
    dx = F.fattn_rope_bwd(wd, t, positions=torch.from_numpy(at).cuda(), interleaved=interleaved).float().cpu().numpy()
    ok()
    x = r.standard_normal((B, H, N, d))


    def f(z):
        return float((w.astype(np.float64) * oracle.rope.rotate(z, ang, interleaved, mag)).sum())

    num = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = 1.0
        num[i] = (f(x + e) - f(x - e)) / 2      # linear: no error but 64-bit rounding
    allow = 2.0 ** -8 * np.abs(num) + 8 * 2.0 ** -24 * np.abs(w).max() * mag + 1e-9
    assert (np.abs(dx - num) <= allow).all()


def test_there_and_back_and_through_attention():
    """Rotated queries and keys through the training kernels: scores depend on
    distances only, so moving all positions along changes O by roundings alone; and
    the gradients turned back are those of the unrotated inputs."""
    torch.manual_seed(3)
    B, H, N, d = 1, 2, 96, 64
    q, k, v, do = (torch.randn(B, H, N, d, device="cuda").to(torch.bfloat16) for _ in range(4))
    t = F.fattn_rope_table(1000, d)
    outs = []
    for shift in (0, 700):
        pos = torch.arange(shift, shift + N, dtype=torch.int32, device="cuda")
        qr, kr = F.fattn_rope(q, t, positions=pos), F.fattn_rope(k, t, positions=pos)
        o, lse = F.fattn_fwd(qr, kr, v, causal=True)
        dq, dk, dv = F.fattn_bwd(qr, kr, v, o, do, lse, causal=True)
        outs.append((o, F.fattn_rope_bwd(dq, t, positions=pos), F.fattn_rope_bwd(dk, t, positions=pos), dv))
    ok()
    # the same in 64 bits on the unrotated inputs, differentiated by torch
    x = [a.double().requires_grad_() for a in (q, k, v)]
    ang = torch.arange(N, device="cuda")[:, None] * torch.from_numpy(oracle.rope.frequencies(d)).cuda()

    def turn(a):
        a0, a1 = a[..., :d // 2], a[..., d // 2:]
        return torch.cat([a0 * ang.cos() - a1 * ang.sin(), a1 * ang.cos() + a0 * ang.sin()], dim=-1)

    s = turn(x[0]) @ turn(x[1]).transpose(2, 3) / d ** 0.5
    s = s.masked_fill(torch.ones(N, N, device="cuda").triu(1).bool(), -torch.inf)
    o = torch.softmax(s, -1) @ x[2]
    o.backward(do.double())
    o = o.detach()
    for got in outs:
        # the training kernels' tolerances: 1e-2 for O, 5e-2 of the largest gradient
        assert float((got[0].double() - o).abs().max()) <= 1e-2
        for g, a in zip(got[1:], x):
            assert float((g.double() - a.grad).abs().max()) <= 5e-2 * float(a.grad.abs().max())


def test_captured_and_on_another_stream():
    x, xd = make(15, (2, 4, 130, 64))
    t = F.fattn_rope_table(200, 64)
    pos = torch.arange(130, dtype=torch.int32, device="cuda")
    want = F.fattn_rope(xd, t, positions=pos + 50)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = F.fattn_rope(xd, t, positions=pos + 50)
    s.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = F.fattn_rope(xd, t, positions=pos)
    pos += 50
    g.replay()
    ok()
    assert torch.equal(y, want)


def test_more_than_32_bits_of_elements():
    """Rows whose offsets pass 2^31 elements."""
    n, d = (1 << 31) // (64 * 2048) + 3, 64
    x = torch.zeros((n, 2048, d), dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.randn(2048, d, device="cuda").to(torch.bfloat16)
    x[0] = x[-1]
    t = F.fattn_rope_table(5, d)
    pos = torch.full((n,), 3, dtype=torch.int32, device="cuda")
    F.fattn_rope(x, t, positions=pos, out=x)
    ok()
    assert torch.equal(x[0], x[-1])
    want = F.fattn_rope(x[:1], F.fattn_rope_table(5, d), positions=pos[:1])
    assert want.shape == (1, 2048, d) and not bool((x[-2] != 0).any())


def test_refusals_of_the_binding():
    x = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16, device="cuda")
    t = F.fattn_rope_table(4, 64)
    for bad in (dict(x=x.float()), dict(x=x[0, 0]), dict(x=x.cpu()), dict(rope=t.double()), dict(rope=t.t()),
                dict(positions=torch.zeros(4, dtype=torch.int32, device="cuda")),
                dict(positions=torch.zeros(3, device="cuda")), dict(out=x[:, :1]), dict(x=x[..., ::2])):
        a = dict(x=x, rope=t, positions=None, out=None)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            F.fattn_rope(a["x"], a["rope"], positions=a["positions"], out=a["out"])
    for shape in ((0, 2, 3, 64), (1, 2, 0, 64)):
        assert F.fattn_rope(torch.zeros(shape, dtype=torch.bfloat16, device="cuda"), t).shape == shape
    with pytest.raises(_lib.FattnError):
        F.fattn_rope(torch.zeros((1, 2, 3, 72), dtype=torch.bfloat16, device="cuda"), t)
